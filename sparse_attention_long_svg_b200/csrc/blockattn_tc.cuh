// The many-query kernels of attention over chosen blocks, on the 5th-generation
// tensor cores: 128 rows (the query heads of floor(128/G) neighbouring tokens)
// against the union of their blocks, 64 keys a step.
//
// Neighbouring tokens choose much alike, so that the union of 128 rows stays
// small: 18 blocks of 16 listed for G = 5 on passages of 192 tokens, 136 of 32
// for G = 1.  A row that does not list a block gets weights of zero there.  A
// zero times an infinity or NaN would still reach its accumulator, so a row
// whose result is not finite is computed again, by itself, from its own keys.
#pragma once

#include "blockattn.cuh"

namespace svg {

constexpr int kTcRows = 128, kTcThreads = 224;

// Byte offset of 16-byte chunk c of row r in a 128-byte-swizzled tile of ROWS
// rows: 64-channel halves of 128-byte rows, chunks exchanged by the row's low bits.
template <int ROWS>
__device__ __forceinline__ uint32_t tc_at(int r, int c) {
  return static_cast<uint32_t>((c >> 3) * ROWS * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// Rows [key0, key0 + 64) of a [Nk, D] matrix by one warp; rows from `len` on
// become zeros.
template <int D>
__device__ __forceinline__ void tc_load_tile(uint32_t dst, const __nv_bfloat16 *src, int key0, int len) {
  constexpr int COLS = D / 8, STEP = 32 / COLS;
  const int r0 = lane_id() / COLS, c = lane_id() % COLS;
  const __nv_bfloat16 *from = src + static_cast<int64_t>(key0 + r0) * D + 8 * c;
  if (key0 + kBaTile <= len) {
#pragma unroll
    for (int r = 0; r < kBaTile; r += STEP) cp_async16(dst + tc_at<kBaTile>(r0 + r, c), from + r * D, 16);
  } else {
#pragma unroll
    for (int r = 0; r < kBaTile; r += STEP) {
      const bool in = key0 + r0 + r < len;
      cp_async16(dst + tc_at<kBaTile>(r0 + r, c), in ? from + r * D : src, in ? 16u : 0u);
    }
  }
}

// A 128-row operand tile (row r of the CTA = row(r) of a [rows, D] matrix, -1:
// zeros) by all threads.
template <int D, typename F>
__device__ __forceinline__ void tc_load_rows(uint32_t dst, const __nv_bfloat16 *src, F row) {
  constexpr int COLS = D / 8;
  for (int i = threadIdx.x; i < kTcRows * COLS; i += kTcThreads) {
    const int r = i / COLS, c = i % COLS;
    const int64_t at = row(r);
    cp_async16(dst + tc_at<kTcRows>(r, c), src + (at >= 0 ? at * D + 8 * c : 0), at >= 0 ? 16u : 0u);
  }
}

struct TcBars {                       // at most 192 bytes
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], done, drain;
  uint32_t tmem;
  int count;
};

__device__ __forceinline__ bool tc_wait(uint64_t *bar, uint32_t parity, uint64_t ns) {
  if (mbar_wait(bar, parity, ns)) return true;
  record_error(SVG_ERR_TIMEOUT, SVG_SITE_BLOCK_ATTN);
  return false;
}
__device__ __forceinline__ bool tc_warp_wait(uint64_t *bar, uint32_t parity, uint64_t ns) {
  const bool ok = mbar_wait(bar, parity, ns);
  if (!ok && lane_id() == 0) record_error(SVG_ERR_TIMEOUT, SVG_SITE_BLOCK_ATTN);
  return __all_sync(0xffffffffu, ok);
}

// Shared memory of the two query-major kernels: `operands` 128-row tiles, two
// stages of K and V, barriers, bit sets, block list.
template <int D>
__host__ __device__ inline size_t tc_smem(int operands, int tokens, int nblk) {
  return static_cast<size_t>(operands) * kTcRows * D * 2 + 4ull * kBaTile * D * 2 + 192 + mark_bytes(tokens, nblk);
}

__device__ __forceinline__ float dot_rows(const __nv_bfloat16 *a, const __nv_bfloat16 *b, int D) {
  float s = 0.f;
  for (int c = 0; c < D; c += 8) {
    float x[8], y[8];
    unpack8(*reinterpret_cast<const uint4 *>(a + c), x);
    unpack8(*reinterpret_cast<const uint4 *>(b + c), y);
#pragma unroll
    for (int e = 0; e < 8; ++e) s += x[e] * y[e];
  }
  return s;
}

// What the CTA's rows share, for the row that is computed again: tiles [u0, u1)
// of the union (key(u)), the row's bit set.
struct TcUnion {
  const uint16_t *list;
  const uint32_t *bits;
  int u0, u1, shift, tokens;           // a block has 2^shift tiles of 64 keys
  __device__ __forceinline__ int block_of(int u) const { return list[u >> shift]; }
  __device__ __forceinline__ int key(int u) const {
    return ((block_of(u) << shift) + (u & ((1 << shift) - 1))) * kBaTile;
  }
  __device__ __forceinline__ bool listed(int tok, int u) const {
    const int j = block_of(u);
    return (bits[(j >> 5) * tokens + tok] >> (j & 31)) & 1u;
  }
};

// One row by one warp, from its own keys alone: two passes over the scores.
// Lane i ends with channels i * D/32 ... of the normalised output.
template <int D>
__device__ __noinline__ void row_again(const TcUnion &un, const __nv_bfloat16 *q, const __nv_bfloat16 *k,
                                       const __nv_bfloat16 *v, int tok, int seen, float sl2, float (&y)[D / 32],
                                       float &lse2) {
  constexpr int E = D / 32;
  const int lane = lane_id();
  float m = -INFINITY, l = 0.f;
  bool nan = false;
#pragma unroll
  for (int e = 0; e < E; ++e) y[e] = 0.f;
  for (int pass = 0; pass < 2; ++pass) {
    for (int u = un.u0; u < un.u1; ++u) {
      if (!un.listed(tok, u)) continue;
      const int key0 = un.key(u), end = min(seen - key0, kBaTile);
      for (int j0 = 0; j0 < end; j0 += 32) {
        const bool in = j0 + lane < end;
        float s = -INFINITY;
        if (in) s = dot_rows(q, k + static_cast<int64_t>(key0 + j0 + lane) * D, D) * sl2;
        if (pass == 0) {
          m = fmaxf(m, s);
          nan = nan || s != s;
          continue;
        }
        const float p = in ? ex2_approx(s - m) : 0.f;
        l += p;
        for (int j = 0; j < min(32, end - j0); ++j) {
          const float pj = __shfl_sync(0xffffffffu, p, j);
          const __nv_bfloat16 *vr = v + static_cast<int64_t>(key0 + j0 + j) * D + lane * E;
#pragma unroll
          for (int e = 0; e < E; ++e) y[e] += pj * __bfloat162float(vr[e]);
        }
      }
    }
    if (pass == 0) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (__any_sync(0xffffffffu, nan)) m = __int_as_float(0x7FC00000);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  // scores of minus infinity only: as without keys
  const float inv = m == -INFINITY ? 0.f : 1.f / l;
#pragma unroll
  for (int e = 0; e < E; ++e) y[e] = m == -INFINITY ? 0.f : y[e] * inv;
  lse2 = m == -INFINITY ? -INFINITY : m + log2f(l);
}

// Warps 0-3: softmax (thread = row = TMEM lane); warp 4: its lane 0 issues the
// matrix products; warp 5 loads K, warp 6 V (two stages each: a K tile is free
// again before the weights of its scores are).  Two score buffers in TMEM; a row's
// weights replace its scores there (bf16, the A operand of the product with V).
//   S(t+1) is issued before P(t) V, so the tensor cores run while the softmax
//   of the other buffer (or of the SM's other CTA) does.
// The reference maximum of a row is raised only when a score exceeds it by 2^8;
// then the accumulator in TMEM is rescaled.
template <int D>
__global__ void __launch_bounds__(kTcThreads, 2) block_attn_tc_kernel(const BlockAttnArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  constexpr int Q_BYTES = kTcRows * D * 2, KV = kBaTile * D * 2, COLS = 256;
  constexpr uint32_t IDESC_S = idesc_bf16_f32(kTcRows, kBaTile, false, false);
  constexpr uint32_t IDESC_PV = idesc_bf16_f32(kTcRows, D, false, true);
  constexpr uint32_t TM_S = D;                      // O, then two score buffers
  constexpr float kRaise = 8.f;
  uint8_t *sKV = smem + Q_BYTES;                    // [stage][K, V]
  TcBars *B = reinterpret_cast<TcBars *>(sKV + 4 * KV);
  uint32_t *bits = reinterpret_cast<uint32_t *>(sKV + 4 * KV + 192);
  const int tokens = kTcRows / a.G;
  const int W = (a.nblk + 31) / 32;
  uint32_t *uni = bits + tokens * W;
  uint16_t *list = reinterpret_cast<uint16_t *>(uni + W);
  const int ntiles = (a.Nq + tokens - 1) / tokens;
  const int head = blockIdx.x / ntiles;             // one head after the other: its K and V stay in L2
  const int n0 = (ntiles - 1 - static_cast<int>(blockIdx.x % ntiles)) * tokens;
  const int len = seq_len(a.kv_len, head / a.heads_per_seq, a.Nk);
  const int warp = warp_id(), lane = lane_id();
  const uint64_t ns = a.wait_ns;

  // row r: head r % G of token n0 + r / G
  auto row_of = [&](int r) -> int64_t {
    const int n = n0 + r / a.G;
    return r < tokens * a.G && n < a.Nq ? (static_cast<int64_t>(head) * a.G + r % a.G) * a.Nq + n : -1;
  };
  if (warp == 4) {
    tmem_alloc(&B->tmem, COLS);
    tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B->k_full[i], 32);
      mbar_init(&B->k_empty[i], 1);
      mbar_init(&B->v_full[i], 32);
      mbar_init(&B->v_empty[i], 1);
      mbar_init(&B->s_full[i], 1);
      mbar_init(&B->p_full[i], 128);
    }
    mbar_init(&B->done, 1);
    mbar_init(&B->drain, 1);
    fence_mbar_init();
  }
  tc_load_rows<D>(smem_u32(smem), a.q, row_of);
  cp_async_commit();
  TcUnion un;
  un.list = list;
  un.bits = bits;
  un.shift = a.block == kBaTile ? 0 : 1;
  un.tokens = tokens;
  tc_fence_before();
  const int total = mark_blocks(a, head, len, n0, tokens, W, bits, uni, list, &B->count) << un.shift;
  tc_fence_after();
  cp_async_wait<0>();
  fence_proxy_async_smem();
  __syncthreads();
  const uint32_t tmem = B->tmem;
  const int each = (total + a.splits - 1) / a.splits;
  un.u0 = min(static_cast<int>(blockIdx.y) * each, total);
  un.u1 = min(un.u0 + each, total);
  const int steps = un.u1 - un.u0;
  const __nv_bfloat16 *kh = a.k + static_cast<int64_t>(head) * a.Nk * D;
  const __nv_bfloat16 *vh = a.v + static_cast<int64_t>(head) * a.Nk * D;

  if (warp >= 5) {
    // ---------------------------------------------------------------- loads: K, V
    const bool is_v = warp == 6;
    uint64_t *full = is_v ? B->v_full : B->k_full, *empty = is_v ? B->v_empty : B->k_empty;
    for (int t = 0; t < steps; ++t) {
      const int st = t & 1;
      if (t >= 2 && !tc_warp_wait(&empty[st], ((t >> 1) - 1) & 1, ns)) break;
      tc_load_tile<D>(smem_u32(sKV) + static_cast<uint32_t>(2 * st + is_v) * KV, is_v ? vh : kh, un.key(un.u0 + t), len);
      cp_async_arrive(&full[st]);
    }
    cp_async_commit();
    cp_async_wait<0>();
  } else if (warp == 4) {
    // ---------------------------------------------------------------- matrix products
    if (lane == 0) {
      const SmemDesc qd = make_desc_sw128(smem_u32(smem), 16, 1024);
      const SmemDesc kd = make_desc_sw128(smem_u32(sKV), 16, 1024);
      const SmemDesc vd = make_desc_sw128(smem_u32(sKV) + KV, kBaTile * 128, 1024);
      auto issue_s = [&](int t) {
        const int st = t & 1;
        if (!tc_wait(&B->k_full[st], (t >> 1) & 1, ns)) return false;
        fence_proxy_async_smem();                   // cp.async writes -> tensor-core reads
        tc_fence_after();
        const uint32_t off = static_cast<uint32_t>(st * 2 * KV) >> 4;
        mma_chain<D / 16, kTcRows * 128, 32, kBaTile * 128, 32>(tmem + TM_S + st * kBaTile, qd,
                                                                SmemDesc{kd.lo + off, kd.hi}, IDESC_S, 0u);
        mma_commit(&B->s_full[st]);
        mma_commit(&B->k_empty[st]);
        return true;
      };
      bool ok = steps == 0 || issue_s(0);
      for (int t = 0; t < steps && ok; ++t) {
        const int st = t & 1;
        // its score buffer held P(t-1), whose product was issued before
        if (t + 1 < steps && !issue_s(t + 1)) break;
        if (!tc_wait(&B->v_full[st], (t >> 1) & 1, ns) || !tc_wait(&B->p_full[st], (t >> 1) & 1, ns)) break;
        fence_proxy_async_smem();
        tc_fence_after();
        const uint32_t off = static_cast<uint32_t>(st * 2 * KV) >> 4;
#pragma unroll
        for (int k = 0; k < kBaTile / 16; ++k)
          mma_bf16_ts(tmem, tmem + TM_S + st * kBaTile + 8 * k,
                      (static_cast<uint64_t>(vd.hi) << 32) | (vd.lo + off + ((k * 2048) >> 4)), IDESC_PV,
                      t > 0 || k > 0 ? 1u : 0u);
        mma_commit(&B->v_empty[st]);
        mma_commit(&B->done);
      }
      mma_commit(&B->drain);                        // all retired before TMEM is released
      mbar_wait(&B->drain, 0, 1000000000ull);
    }
  } else {
    // ---------------------------------------------------------------- softmax
    const int r = warp * 32 + lane;
    const int64_t row = row_of(r);
    const int tok = row >= 0 ? r / a.G : 0;
    const int seen = row >= 0 ? query_seen(a, len, n0 + tok) : 0;
    const uint32_t mine = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int t = 0; t < steps; ++t) {
      const int st = t & 1, u = un.u0 + t;
      const int key0 = un.key(u);
      const int end = row >= 0 && un.listed(tok, u) ? seen - key0 : 0;
      const uint32_t s_at = mine + TM_S + st * kBaTile;
      if (!tc_warp_wait(&B->s_full[st], (t >> 1) & 1, ns)) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (!__any_sync(0xffffffffu, end > 0)) {      // none of the warp's rows lists the block
        float p[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) p[c] = 0.f;
        tmem_st32(s_at, p);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&B->p_full[st]);
        continue;
      }
      float s[64];
      tmem_ld64_sync(s_at, s);
      if (__any_sync(0xffffffffu, end > 0 && end < kBaTile)) {
#pragma unroll
        for (int c = 0; c < 64; ++c) s[c] = c < end ? s[c] : -INFINITY;
      }
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int c = 0; c < 64; c += 2) mx[(c >> 1) & 3] = max3f(mx[(c >> 1) & 3], s[c], s[c + 1]);
      const float top = end > 0 ? fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2 : -INFINITY;
      float f = 1.f;
      if (top > m + kRaise) {                       // also the row's first block (m = -inf, nothing to rescale)
        if (m > -INFINITY) f = ex2_approx(m - top);
        m = top;
      }
      if (__any_sync(0xffffffffu, f != 1.f)) {
        // S(t) complete implies P(t-2) V complete, so this phase is at most one behind
        if (!tc_warp_wait(&B->done, (t - 1) & 1, ns)) {
          ok = false;
          break;
        }
        tc_fence_after();
        l *= f;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
          tmem_ld32_sync(mine + c, o);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] *= f;
          tmem_st32(mine + c, o);
        }
      }
      // a row without keys here: minus infinity, weights of zero; others are 2^8 at most
      const float base = end > 0 && m > -INFINITY ? -m : -INFINITY;
      const float2 sc = make_float2(a.scale_log2, a.scale_log2), nm = make_float2(base, base);
      float2 sum = make_float2(0.f, 0.f);
      float p[32];
#pragma unroll
      for (int c = 0; c < 64; c += 2) {
        const float2 x = fma_f32x2(make_float2(s[c], s[c + 1]), sc, nm);
        const float2 w = make_float2(ex2_approx(x.x), ex2_approx(x.y));
        sum = add_f32x2(sum, w);
        // weights as bf16 for the matrix product: 2^-8 relative to each; the sum keeps fp32
        p[c >> 1] = __uint_as_float(pack_bf16x2(w.x, w.y));
      }
      l += sum.x + sum.y;
      tmem_st32(s_at, p);
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&B->p_full[st]);
    }
    if (ok && steps > 0) ok = tc_warp_wait(&B->done, (steps - 1) & 1, ns);
    tc_fence_after();
    const bool none = m == -INFINITY && l == 0.f;
    const float inv = none ? 0.f : 1.f / l;
    float lse2 = none ? -INFINITY : m + log2f(l);
    const int64_t part = static_cast<int64_t>(blockIdx.y) * a.BHk * a.G * a.Nq + row;
    // a timeout leaves the outputs undefined
    bool bad = row >= 0 && !none && !(fabsf(lse2) < INFINITY);
    if (ok && steps > 0) {
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        float o[32];
        tmem_ld32_sync(mine + c, o);
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          bad = bad || (!none && !(fabsf(o[e]) < INFINITY));
          o[e] = none ? 0.f : o[e] * inv;
        }
        if (row >= 0) {
          if (a.splits > 1) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<float4 *>(a.part_o + part * D + c + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          } else {
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              float y[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) y[i] = o[e + i];
              *reinterpret_cast<uint4 *>(a.o + row * D + c + e) = pack8(y);
            }
          }
        }
      }
    } else if (row >= 0) {
      for (int c = 0; c < D; c += 8) {
        if (a.splits > 1) {
          *reinterpret_cast<float4 *>(a.part_o + part * D + c) = make_float4(0, 0, 0, 0);
          *reinterpret_cast<float4 *>(a.part_o + part * D + c + 4) = make_float4(0, 0, 0, 0);
        } else {
          *reinterpret_cast<uint4 *>(a.o + row * D + c) = make_uint4(0, 0, 0, 0);
        }
      }
    }
    for (uint32_t again = __ballot_sync(0xffffffffu, ok && row >= 0 && bad); again; again &= again - 1) {
      const int src = __ffs(again) - 1;
      const int64_t rw = __shfl_sync(0xffffffffu, row, src);
      float y[D / 32], z;
      row_again<D>(un, a.q + rw * D, kh, vh, __shfl_sync(0xffffffffu, tok, src), __shfl_sync(0xffffffffu, seen, src),
                   a.scale_log2, y, z);
      const int64_t pr = __shfl_sync(0xffffffffu, part, src);
#pragma unroll
      for (int e = 0; e < D / 32; e += 2) {
        if (a.splits > 1)
          *reinterpret_cast<float2 *>(a.part_o + pr * D + lane * (D / 32) + e) = make_float2(y[e], y[e + 1]);
        else
          *reinterpret_cast<uint32_t *>(a.o + rw * D + lane * (D / 32) + e) = pack_bf16(y[e], y[e + 1]);
      }
      if (lane == src) lse2 = z;
    }
    if (row >= 0) {
      if (a.splits > 1)
        a.part_lse[part] = lse2;
      else if (a.lse)
        a.lse[row] = lse2 * 0.69314718055994531f;
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc(tmem, COLS);
  }
}

}  // namespace svg
