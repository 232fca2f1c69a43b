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

// Row r < 128 of a tile: head r % G of token n0 + r / G, as a row of
// [BHk*G, Nq] (-1: none).  The reciprocal of G is exact enough for r < 128.
struct TcRowMap {
  uint32_t per;
  int G, n0, rows, Nq;
  int64_t base;
  __device__ __forceinline__ TcRowMap(const BlockAttnArgs &a, int head, int n0_, int tokens)
      : per(65535u / a.G + 1), G(a.G), n0(n0_), rows(min(tokens, a.Nq - n0_) * a.G), Nq(a.Nq),
        base(static_cast<int64_t>(head) * a.G * a.Nq) {}
  __device__ __forceinline__ int token(int r) const { return static_cast<int>((r * per) >> 16); }
  __device__ __forceinline__ int64_t operator()(int r) const {
    const int t = token(r);
    return r < rows ? base + static_cast<int64_t>(r - t * G) * Nq + n0 + t : -1;
  }
};

// A 128-row operand tile (row r of the CTA = row(r) of a [rows, D] matrix, -1:
// zeros) by all threads.
template <int D, int THREADS, typename F>
__device__ __forceinline__ void tc_load_rows(uint32_t dst, const __nv_bfloat16 *src, F row) {
  constexpr int COLS = D / 8;
#pragma unroll
  for (int i0 = 0; i0 < kTcRows * COLS; i0 += THREADS) {
    const int i = i0 + threadIdx.x, r = i / COLS, c = i % COLS;
    if (i >= kTcRows * COLS) break;
    const int64_t at = row(r);
    cp_async16(dst + tc_at<kTcRows>(r, c), src + (at >= 0 ? at * D + 8 * c : 0), at >= 0 ? 16u : 0u);
  }
}

// The issuing warp runs as a whole, with one elected lane behind a predicate of
// each instruction: operands then are uniform registers.  Issued from a branch
// that one lane takes, every descriptor word goes through a move to one, about
// 80 clocks for each of these short products.
__device__ __forceinline__ void tc_mma_ss(uint32_t d, SmemDesc a, uint32_t a_off, SmemDesc b, uint32_t b_off,
                                          uint32_t idesc, uint32_t accumulate, uint32_t elected) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 ad, bd;\n\t"
      "mov.b64 ad, {%1, %2};\n\tmov.b64 bd, {%3, %4};\n\t"
      "setp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 e, %7, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], ad, bd, %5, p;\n\t}" ::"r"(d),
      "r"(a.lo + a_off), "r"(a.hi), "r"(b.lo + b_off), "r"(b.hi), "r"(idesc), "r"(accumulate), "r"(elected)
      : "memory");
}
// A from TMEM (lane = row, two bf16 per column).
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, SmemDesc b, uint32_t b_off, uint32_t idesc,
                                          uint32_t accumulate, uint32_t elected) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 bd;\n\t"
      "mov.b64 bd, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 e, %6, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], bd, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b.lo + b_off), "r"(b.hi), "r"(idesc), "r"(accumulate), "r"(elected)
      : "memory");
}
__device__ __forceinline__ void tc_commit(uint64_t *bar, uint32_t elected) {
  asm volatile(
      "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(elected)
      : "memory");
}
// K16 steps into one accumulator: step k lies (k / 4) * X_HALF + (k % 4) * X_K bytes behind the operand's start.
template <int STEPS, uint32_t A_HALF, uint32_t A_K, uint32_t B_HALF, uint32_t B_K>
__device__ __forceinline__ void tc_chain(uint32_t d, SmemDesc a, SmemDesc b, uint32_t idesc, uint32_t accumulate_first,
                                         uint32_t elected) {
#pragma unroll
  for (int k = 0; k < STEPS; ++k)
    tc_mma_ss(d, a, ((k >> 2) * A_HALF + (k & 3) * A_K) >> 4, b, ((k >> 2) * B_HALF + (k & 3) * B_K) >> 4, idesc,
              k > 0 ? 1u : accumulate_first, elected);
}

struct TcBars {                       // at most 192 bytes
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], done, last, drain;
  uint32_t tmem;
  int count;
};

__device__ __forceinline__ bool tc_warp_wait(uint64_t *bar, uint32_t parity, uint64_t ns) {
  const bool ok = mbar_wait(bar, parity, ns);
  if (!ok && lane_id() == 0) record_error(SVG_ERR_TIMEOUT, SVG_SITE_BLOCK_ATTN);
  return __all_sync(0xffffffffu, ok);
}

// Shared memory of the forward kernel: `operands` 128-row tiles, two
// stages of K and V, barriers, bit sets, block list.
template <int D>
__host__ __device__ constexpr size_t tc_smem(int operands, int tokens, int nblk) {
  return static_cast<size_t>(operands) * kTcRows * D * 2 + 4ull * kBaTile * D * 2 + 192 + mark_bytes(tokens, nblk);
}

// Warps 0-3: softmax (thread = row = TMEM lane); warp 4: its lane 0 issues the
// matrix products; warp 5 loads K, warp 6 V (two stages each: a K tile is free
// again before the weights of its scores are).  Two score buffers in TMEM; a row's
// weights replace its scores there (bf16, the A operand of the product with V).
//   S(t+1) is issued before P(t) V, so the tensor cores run while the softmax
//   of the other buffer (or of the SM's other CTA) does.
// The reference maximum of a row is raised only when a score exceeds it by 2^8;
// then the accumulator in TMEM is rescaled.  A step moves 96 KB through shared
// memory (the short products read their operands from there), 770 of the about
// 900 clocks it takes per SM: 500 us for 2 x 8,190 tokens, 40 / 8 heads, 16 blocks
// (545 TFLOP/s of listed work), 1,190 us for 8 x 32,760 tokens, 32 blocks.
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
  const int tokens = a.tile_tokens;
  const int W = (a.nblk + 31) / 32;
  uint32_t *uni = bits + tokens * W;
  uint16_t *list = reinterpret_cast<uint16_t *>(uni + W);
  const int ntiles = (a.Nq + tokens - 1) / tokens;
  const int head = blockIdx.x / ntiles;             // one head after the other: its K and V stay in L2
  const int n0 = (ntiles - 1 - static_cast<int>(blockIdx.x % ntiles)) * tokens;
  const int len = seq_len(a.kv_len, head / a.heads_per_seq, a.Nk);
  const int warp = warp_id(), lane = lane_id();
  const uint64_t ns = a.wait_ns;
  const TcRowMap row_of(a, head, n0, tokens);
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
    mbar_init(&B->last, 1);
    mbar_init(&B->drain, 1);
    fence_mbar_init();
  }
  tc_load_rows<D, kTcThreads>(smem_u32(smem), a.q, row_of);
  cp_async_commit();
  BaUnion un;
  un.list = list;
  un.bits = bits;
  un.keys = kBaTile;
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
    for (int t = 0; t < steps && !a.fault; ++t) {
      const int st = t & 1;
      if (t >= 2 && !tc_warp_wait(&empty[st], ((t >> 1) - 1) & 1, ns)) break;
      tc_load_tile<D>(smem_u32(sKV) + static_cast<uint32_t>(2 * st + is_v) * KV, is_v ? vh : kh, un.key(un.u0 + t), len);
      cp_async_arrive(&full[st]);
    }
    cp_async_commit();
    cp_async_wait<0>();
  } else if (warp == 4) {
    // ---------------------------------------------------------------- matrix products
    {
      const uint32_t el = elect_one();
      const SmemDesc qd = make_desc_sw128(smem_u32(smem), 16, 1024);
      const SmemDesc kd = make_desc_sw128(smem_u32(sKV), 16, 1024);
      const SmemDesc vd = make_desc_sw128(smem_u32(sKV) + KV, kBaTile * 128, 1024);
      int n_s = 0;                                  // score products issued
      auto issue_s = [&]() {
        const int st = n_s & 1;
        if (!tc_warp_wait(&B->k_full[st], (n_s >> 1) & 1, ns)) return false;
        fence_proxy_async_smem();                   // cp.async writes -> tensor-core reads
        tc_fence_after();
        const uint32_t off = static_cast<uint32_t>(st * 2 * KV) >> 4;
        tc_chain<D / 16, kTcRows * 128, 32, kBaTile * 128, 32>(tmem + TM_S + st * kBaTile, qd,
                                                                SmemDesc{kd.lo + off, kd.hi}, IDESC_S, 0u, el);
        tc_commit(&B->s_full[st], el);
        tc_commit(&B->k_empty[st], el);
        ++n_s;
        return true;
      };
      bool ok = steps == 0 || issue_s();
      for (int t = 0; t < steps && ok; ++t) {
        const int st = t & 1;
        // its score buffer held P(t-1), whose product was issued before
        if (t + 1 < steps && !issue_s()) break;
        if (!tc_warp_wait(&B->v_full[st], (t >> 1) & 1, ns) || !tc_warp_wait(&B->p_full[st], (t >> 1) & 1, ns)) break;
        fence_proxy_async_smem();
        tc_fence_after();
        const uint32_t off = static_cast<uint32_t>(st * 2 * KV) >> 4;
#pragma unroll
        for (int k = 0; k < kBaTile / 16; ++k)
          tc_mma_ts(tmem, tmem + TM_S + st * kBaTile + 8 * k, vd, off + ((k * 2048) >> 4), IDESC_PV,
                    t > 0 || k > 0 ? 1u : 0u, el);
        tc_commit(&B->v_empty[st], el);
        tc_commit(&B->done, el);
        if (t == steps - 1) tc_commit(&B->last, el);
      }
      tc_commit(&B->drain, el);                        // all retired before TMEM is released
      mbar_wait(&B->drain, 0, 1000000000ull);
    }
  } else {
    // ---------------------------------------------------------------- softmax
    const int r = warp * 32 + lane;
    const int64_t row = row_of(r);
    const int tok = row >= 0 ? row_of.token(r) : 0;
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
    // (`done` may still be two phases behind here, where its parity would tell nothing)
    if (ok && steps > 0) ok = tc_warp_wait(&B->last, 0, ns);
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


// ------------------------------------------------------------------ gradient
// One row of dQ by one warp, from its own keys alone (see row_again).
template <int D>
__device__ __noinline__ void dq_row_again(const BaUnion &un, const __nv_bfloat16 *q, const __nv_bfloat16 *dout,
                                          const __nv_bfloat16 *k, const __nv_bfloat16 *v, int tok, int seen, float sl2,
                                          float lse2, float delta, float (&y)[D / 32]) {
  constexpr int E = D / 32;
  const int lane = lane_id();
#pragma unroll
  for (int e = 0; e < E; ++e) y[e] = 0.f;
  for (int u = un.u0; u < un.u1; ++u) {
    if (!un.listed(tok, u)) continue;
    const int key0 = un.key(u), end = min(seen - key0, un.keys);
    for (int j0 = 0; j0 < end; j0 += 32) {
      float ds = 0.f;
      if (j0 + lane < end) {
        const int64_t at = static_cast<int64_t>(key0 + j0 + lane) * D;
        ds = ex2_approx(dot_rows(q, k + at, D) * sl2 - lse2) * (dot_rows(dout, v + at, D) - delta);
      }
      for (int j = 0; j < min(32, end - j0); ++j) {
        const float g = __shfl_sync(0xffffffffu, ds, j);
        const __nv_bfloat16 *kr = k + static_cast<int64_t>(key0 + j0 + j) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) y[e] += g * __bfloat162float(kr[e]);
      }
    }
  }
}

// 16 consecutive fp32 columns of this thread's TMEM lane, waited for inside the
// same asm statement.
__device__ __forceinline__ void tmem_ld16_sync(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// dQ, and delta for the second kernel: 128 rows against their union, as in the
// forward kernel.  A step is a chain (K, V -> S, dP -> dS -> dQ), and a list is
// short beside a CTA's start-up, so everything is held once and two CTAs share
// an SM: one's chain and start-up fill the other's gaps (one CTA with three
// stages and two score buffers took 650 us where this takes 470: 8,190 tokens,
// 40 / 8 heads, 16 blocks).  Warps 0-7: two groups, 32 keys of a step each (a
// TMEM lane belongs to a thread of each); a group's dS replaces its own scores
// there, as the A operand of the product with K; warp 8 issues, 9 and 10 load.
constexpr int kTcDqThreads = 11 * 32;

struct TcDqBars {                      // at most 128 bytes
  uint64_t k_full[2], k_empty[2], v_full, v_empty, s_full, ds_full, done, drain;
  uint32_t tmem;
  int count;
};

template <int D>
__host__ __device__ constexpr size_t tc_dq_smem(int k_stages, int tokens, int nblk) {
  return 2ull * kTcRows * D * 2 + (1ull + k_stages) * kBaTile * D * 2 + 128 + mark_bytes(tokens, nblk);
}

template <int D>
__global__ void __launch_bounds__(kTcDqThreads, 2) block_attn_dq_tc_kernel(const BlockAttnArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  constexpr int Q_BYTES = kTcRows * D * 2, KV = kBaTile * D * 2, COLS = 256;
  constexpr uint32_t IDESC_S = idesc_bf16_f32(kTcRows, kBaTile, false, false);
  constexpr uint32_t IDESC_DQ = idesc_bf16_f32(kTcRows, D, false, true);
  constexpr uint32_t TM_S = D, TM_DP = D + kBaTile;
  uint8_t *sV = smem + 2 * Q_BYTES, *sK = sV + KV;      // K: one or two stages
  const int NK = a.k_stages;
  TcDqBars *B = reinterpret_cast<TcDqBars *>(sK + NK * KV);
  uint32_t *bits = reinterpret_cast<uint32_t *>(sK + NK * KV + 128);
  const int tokens = a.tile_tokens;
  const int W = (a.nblk + 31) / 32;
  uint32_t *uni = bits + tokens * W;
  uint16_t *list = reinterpret_cast<uint16_t *>(uni + W);
  const int ntiles = (a.Nq + tokens - 1) / tokens;
  const int head = blockIdx.x / ntiles;
  const int n0 = (ntiles - 1 - static_cast<int>(blockIdx.x % ntiles)) * tokens;
  const int len = seq_len(a.kv_len, head / a.heads_per_seq, a.Nk);
  const int warp = warp_id(), lane = lane_id();
  const uint64_t ns = a.wait_ns;
  const TcRowMap row_of(a, head, n0, tokens);
  if (warp == 8) {
    tmem_alloc(&B->tmem, COLS);
    tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B->k_full[i], 32);
      mbar_init(&B->k_empty[i], 1);
    }
    mbar_init(&B->v_full, 32);
    mbar_init(&B->v_empty, 1);
    mbar_init(&B->s_full, 1);
    mbar_init(&B->ds_full, 256);
    mbar_init(&B->done, 1);
    mbar_init(&B->drain, 1);
    fence_mbar_init();
  }
  tc_load_rows<D, kTcDqThreads>(smem_u32(smem), a.q, row_of);
  tc_load_rows<D, kTcDqThreads>(smem_u32(smem) + Q_BYTES, a.dout, row_of);
  cp_async_commit();
  // O for delta: D/8 lanes to a row
  constexpr int OL = (kTcRows * (D / 8) + kTcDqThreads - 1) / kTcDqThreads;
  uint4 o_row[OL];
#pragma unroll
  for (int k = 0; k < OL; ++k) {
    const int i = k * kTcDqThreads + threadIdx.x;
    const int64_t row = i < kTcRows * (D / 8) ? row_of(i / (D / 8)) : -1;
    o_row[k] = row >= 0 ? __ldg(reinterpret_cast<const uint4 *>(a.out + row * D + 8 * (i % (D / 8)))) : make_uint4(0, 0, 0, 0);
  }
  BaUnion un;
  un.list = list;
  un.bits = bits;
  un.keys = kBaTile;
  un.shift = a.block == kBaTile ? 0 : 1;
  un.tokens = tokens;
  un.u0 = 0;
  tc_fence_before();
  un.u1 = mark_blocks(a, head, len, n0, tokens, W, bits, uni, list, &B->count) << un.shift;
  tc_fence_after();
  cp_async_wait<0>();
  fence_proxy_async_smem();
  __syncthreads();
  // delta = rowsum(dO O)
#pragma unroll
  for (int k = 0; k < OL; ++k) {
    const int i = k * kTcDqThreads + threadIdx.x, r = i / (D / 8), c = i % (D / 8);
    if (i >= kTcRows * (D / 8)) break;              // by whole warps
    float x[8], y[8], s = 0.f;
    unpack8(*reinterpret_cast<const uint4 *>(smem + Q_BYTES + tc_at<kTcRows>(r, c)), x);
    unpack8(o_row[k], y);
#pragma unroll
    for (int e = 0; e < 8; ++e) s += x[e] * y[e];
#pragma unroll
    for (int o = D / 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (c == 0) {
      const int64_t row = row_of(r);
      if (row >= 0) a.delta[row] = s;               // read back below, by this CTA, after the barrier
    }
  }
  __syncthreads();
  const uint32_t tmem = B->tmem;
  const int steps = un.u1;
  const __nv_bfloat16 *kh = a.k + static_cast<int64_t>(head) * a.Nk * D;
  const __nv_bfloat16 *vh = a.v + static_cast<int64_t>(head) * a.Nk * D;

  if (warp >= 9) {
    // ---------------------------------------------------------------- loads: K, V
    const bool is_v = warp == 10;
    uint64_t *full = is_v ? &B->v_full : B->k_full, *empty = is_v ? &B->v_empty : B->k_empty;
    const int stages = is_v ? 1 : NK;
    int st = 0, ph = 1;
    for (int t = 0; t < steps && !a.fault; ++t) {
      if (t >= stages && !tc_warp_wait(&empty[st], ph, ns)) break;
      tc_load_tile<D>(smem_u32(is_v ? sV : sK) + static_cast<uint32_t>(st) * KV, is_v ? vh : kh, un.key(t), len);
      cp_async_arrive(&full[st]);
      if (++st == stages) {
        st = 0;
        ph ^= 1;
      }
    }
    cp_async_commit();
    cp_async_wait<0>();
  } else if (warp == 8) {
    // ---------------------------------------------------------------- matrix products
    {
      const uint32_t el = elect_one();
      const SmemDesc qd = make_desc_sw128(smem_u32(smem), 16, 1024);
      const SmemDesc od = make_desc_sw128(smem_u32(smem) + Q_BYTES, 16, 1024);
      const SmemDesc kd = make_desc_sw128(smem_u32(sK), 16, 1024);
      const SmemDesc vd = make_desc_sw128(smem_u32(sV), 16, 1024);
      const SmemDesc kn = make_desc_sw128(smem_u32(sK), kBaTile * 128, 1024);
      int st = 0, ph = 0;                           // K's stage
      for (int t = 0; t < steps; ++t) {
        if (!tc_warp_wait(&B->k_full[st], ph, ns) || !tc_warp_wait(&B->v_full, t & 1, ns)) break;
        const uint32_t off = static_cast<uint32_t>(st * KV) >> 4;
        fence_proxy_async_smem();                   // cp.async writes -> tensor-core reads
        tc_fence_after();
        tc_chain<D / 16, kTcRows * 128, 32, kBaTile * 128, 32>(tmem + TM_S, qd, SmemDesc{kd.lo + off, kd.hi}, IDESC_S,
                                                               0u, el);
        tc_chain<D / 16, kTcRows * 128, 32, kBaTile * 128, 32>(tmem + TM_DP, od, vd, IDESC_S, 0u, el);
        tc_commit(&B->s_full, el);
        tc_commit(&B->v_empty, el);
        if (!tc_warp_wait(&B->ds_full, t & 1, ns)) break;
        tc_fence_after();
        // 16 keys a step; a group's 32 columns hold its high parts, then the low ones
#pragma unroll
        for (int k = 0; k < 2 * kBaTile / 16; ++k) {
          const int j = k & 3;
          tc_mma_ts(tmem, tmem + TM_S + 32 * (j >> 1) + 8 * (j & 1) + (k >= 4 ? 16 : 0), kn, off + ((j * 2048) >> 4),
                    IDESC_DQ, t > 0 || k > 0 ? 1u : 0u, el);
        }
        tc_commit(&B->k_empty[st], el);
        if (t == steps - 1) tc_commit(&B->done, el);
        if (++st == NK) {
          st = 0;
          ph ^= 1;
        }
      }
      tc_commit(&B->drain, el);
      mbar_wait(&B->drain, 0, 1000000000ull);
    }
  } else {
    // ---------------------------------------------------------------- dS
    const int grp = warp >> 2, r = (warp & 3) * 32 + lane;
    const int64_t row = row_of(r);
    const int tok = row >= 0 ? row_of.token(r) : 0;
    const float z = row >= 0 ? __ldg(a.lse_in + row) * 1.4426950408889634f : 0.f, delta = row >= 0 ? a.delta[row] : 0.f;
    // a row without a finite score (lse = -inf) is constant: it sees nothing here
    const int seen = row >= 0 && z != -INFINITY ? query_seen(a, len, n0 + tok) : 0;
    const uint32_t mine = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_at = mine + TM_S + 32 * grp, p_at = mine + TM_DP + 32 * grp;
    bool ok = true;
    for (int t = 0; t < steps; ++t) {
      const int key0 = un.key(t) + 32 * grp;
      const int end = row >= 0 && un.listed(tok, t) ? seen - key0 : 0;
      if (!tc_warp_wait(&B->s_full, t & 1, ns)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const bool any = __any_sync(0xffffffffu, end > 0), part = __any_sync(0xffffffffu, end > 0 && end < 32);
      float g[32];                                  // high parts of 32 keys, low parts
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (any) {
          float s[16], dp[16];
          tmem_ld16_sync(s_at + 16 * h, s);
          tmem_ld16_sync(p_at + 16 * h, dp);
#pragma unroll
          for (int c = 0; c < 16; c += 2) {
            float d[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float p = ex2_approx(fmaf(s[c + e], a.scale_log2, -z));
              d[e] = p * (dp[c + e] - delta);
              if (part) d[e] = 16 * h + c + e < end ? d[e] : 0.f;
            }
            // dS as two bf16 parts (2^-16 relative): a row's dS add up to zero, so what the keys have in common
            // cancels in dQ, and rounding to one part would leave 2.5 times the error
            const uint32_t top = end > 0 ? pack_bf16x2(d[0], d[1]) : 0u;
            g[8 * h + (c >> 1)] = __uint_as_float(top);
            g[16 + 8 * h + (c >> 1)] =
                end > 0 ? __uint_as_float(pack_bf16x2(d[0] - __uint_as_float(top << 16),
                                                      d[1] - __uint_as_float(top & 0xFFFF0000u)))
                        : 0.f;
          }
        } else {
#pragma unroll
          for (int c = 0; c < 8; ++c) g[8 * h + c] = g[16 + 8 * h + c] = 0.f;
        }
      }
      tmem_st32(s_at, g);
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&B->ds_full);
    }
    if (grp == 0) {
      // ---- the accumulator: scaled, stored, rows that are not finite again
      if (ok && steps > 0) ok = tc_warp_wait(&B->done, 0, ns);
      tc_fence_after();
      bool bad = false;
      for (int c = 0; c < D; c += 32) {
        float o[32];
        if (ok && steps > 0) {
          tmem_ld32_sync(mine + c, o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          float y[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            y[i] = o[e + i] * a.scale;
            bad = bad || !(fabsf(y[i]) < INFINITY);
          }
          if (row >= 0) *reinterpret_cast<uint4 *>(a.dq + row * D + c + e) = pack8(y);
        }
      }
      for (uint32_t again = __ballot_sync(0xffffffffu, ok && row >= 0 && bad); again; again &= again - 1) {
        const int src = __ffs(again) - 1;
        const int64_t rw = __shfl_sync(0xffffffffu, row, src);
        float y[D / 32];
        dq_row_again<D>(un, a.q + rw * D, a.dout + rw * D, kh, vh, __shfl_sync(0xffffffffu, tok, src),
                        __shfl_sync(0xffffffffu, seen, src), a.scale_log2, __shfl_sync(0xffffffffu, z, src),
                        __shfl_sync(0xffffffffu, delta, src), y);
#pragma unroll
        for (int e = 0; e < D / 32; e += 2)
          *reinterpret_cast<uint32_t *>(a.dq + rw * D + lane * (D / 32) + e) =
              pack_bf16(y[e] * a.scale, y[e + 1] * a.scale);
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, COLS);
  }
}

// dK and dV of one key tile over one work item's queries (see
// block_attn_count_kernel): 128 gathered (query, head) rows a step.
//   S = Q K^T, dP = dO V^T (rows x keys, double buffered in TMEM)
//   dV^T += dO^T P, dK^T += Q^T dS (channels x keys; P and dS through shared
//   memory, rows of keys, the MN-major B operand)
// D = 64 would leave half of the 128 accumulator lanes empty, so there one
// product [dO | Q]^T [P | dS] makes both (its other two quarters are not read).
// Warps 0-7: two groups, 32 keys each; warp 8: matrix products; warps 9-12: loads.
// A step moves 288 KB through shared memory (operands 192, gathered rows 64, P and
// dS 32), 2,300 of the 3,200 clocks it takes: 650 us for 8,190 tokens, 40 / 8 heads,
// 16 blocks.  Sums of one item stay in TMEM; items of 4,096 rows keep the fp32
// slots of a tile with several at a tenth of the time.
constexpr int kTcDkvThreads = 13 * 32;

struct TcDkvBars {                     // at most 256 bytes
  uint64_t q_full[2], q_empty[2], s_full[2], p_full, p_free, done, drain;
  uint32_t tmem;
  int warp_sum[kTcDkvThreads / 32];
};

template <int D>
__host__ __device__ constexpr size_t tc_dkv_smem(int item_tokens) {
  return 2ull * kBaTile * D * 2 + 4ull * kTcRows * D * 2 + 2ull * kTcRows * 128 + 256 + static_cast<size_t>(item_tokens) * 4;
}

template <int D>
__global__ void __launch_bounds__(kTcDkvThreads, 1) block_attn_dkv_tc_kernel(const BlockAttnArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  constexpr int KV = kBaTile * D * 2, QT = kTcRows * D * 2, PT = kTcRows * 128, COLS = 512;
  constexpr uint32_t IDESC_S = idesc_bf16_f32(kTcRows, kBaTile, false, false);
  constexpr uint32_t IDESC_G = idesc_bf16_f32(128, D == 128 ? kBaTile : 128, true, true);
  constexpr uint32_t TM_S = 0, TM_DP = 128, TM_DV = 256, TM_DK = 320;
  uint8_t *sK = smem, *sV = sK + KV, *sQ = sV + KV;          // [stage][dO, Q]
  uint8_t *sP = sQ + 4 * QT, *sG = sP + PT;
  TcDkvBars *B = reinterpret_cast<TcDkvBars *>(sG + PT);
  int *toks = reinterpret_cast<int *>(sG + PT + 256);
  const int sub = a.block / kBaTile;
  const int tiles = a.BHk * a.nblk * sub;
  const int item = blockIdx.x;
  if (item >= a.item_first[tiles]) return;
  const int tile = a.items[item];
  const int first = a.item_first[tile];
  const bool alone = a.item_first[tile + 1] - first == 1;
  const int64_t blk = tile / sub;
  const int head = static_cast<int>(blk / a.nblk);
  const int key0 = static_cast<int>(blk % a.nblk) * a.block + (tile % sub) * kBaTile;
  const int len = seq_len(a.kv_len, head / a.heads_per_seq, a.Nk);
  const int warp = warp_id(), lane = lane_id();
  const uint64_t ns = a.wait_ns;
  if (warp == 8) {
    tmem_alloc(&B->tmem, COLS);
    tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B->q_full[i], 128);
      mbar_init(&B->q_empty[i], 1);
      mbar_init(&B->s_full[i], 1);
    }
    mbar_init(&B->p_full, 256);
    mbar_init(&B->p_free, 1);
    mbar_init(&B->done, 1);
    mbar_init(&B->drain, 1);
    fence_mbar_init();
  }
  if (warp >= 11) {
    tc_load_tile<D>(smem_u32(warp == 11 ? sK : sV),
                    (warp == 11 ? a.k : a.v) + static_cast<int64_t>(head) * a.Nk * D, key0, len);
    cp_async_commit();
  }
  // this item's queries: places [skip, skip + item_tokens) of the block's bit
  // set; each warp takes a run of its words, counts, then writes
  constexpr int WARPS = kTcDkvThreads / 32;
  const int skip = (item - first) * a.item_tokens;
  const int WQ = (a.Nq + 31) / 32;
  const uint32_t *rev = a.rev + blk * WQ;
  const int run = ((WQ + WARPS - 1) / WARPS + 31) / 32 * 32, w_end = min(WQ, (warp + 1) * run);
  int mine_count = 0;
  for (int w = warp * run + lane; w < w_end; w += 32) mine_count += __popc(__ldg(rev + w));
  mine_count = __reduce_add_sync(0xffffffffu, mine_count);
  if (lane == 0) B->warp_sum[warp] = mine_count;
  __syncthreads();
  int at = -skip, listed = 0;
  for (int i = 0; i < WARPS; ++i) {
    if (i < warp) at += B->warp_sum[i];
    listed += B->warp_sum[i];
  }
  for (int w0 = warp * run; w0 < w_end && at < a.item_tokens; w0 += 32) {
    const uint32_t u = w0 + lane < w_end ? __ldg(rev + w0 + lane) : 0u;
    for (int i = 0; i < 32; ++i) {                  // a lane to a bit
      const uint32_t x = __shfl_sync(0xffffffffu, u, i);
      const int p = at + __popc(x & ((1u << lane) - 1));
      if (((x >> lane) & 1u) && p >= 0 && p < a.item_tokens) toks[p] = (w0 + i) * 32 + lane;
      at += __popc(x);
    }
  }
  cp_async_wait<0>();
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = B->tmem;
  const int rows = min(max(listed - skip, 0), a.item_tokens) * a.G;
  const int steps = (rows + kTcRows - 1) / kTcRows;
  const int64_t qbase = static_cast<int64_t>(head) * a.G * a.Nq;
  // (query, head) row i of the item as a row of [BHk*G*Nq], and its query
  const uint32_t per = 0xFFFFFFFFu / a.G + 1;       // i / G for i < 2^16
  auto source = [&](int i, int &n) {
    const int q = a.G == 1 ? i : static_cast<int>(__umulhi(i, per));
    n = toks[q];
    return qbase + static_cast<int64_t>(i - q * a.G) * a.Nq + n;
  };

  if (warp >= 9) {
    // ---------------------------------------------------------------- loads: 32 rows a warp
    constexpr int COLS16 = D / 8, PER = 32 / COLS16;
    const int base_row = (warp - 9) * 32, c = lane % COLS16;
    for (int t = 0; t < steps && !a.fault; ++t) {
      const int st = t & 1;
      if (t >= 2 && !tc_warp_wait(&B->q_empty[st], ((t >> 1) - 1) & 1, ns)) break;
      const int i = t * kTcRows + base_row + lane;
      int n;
      const int64_t at = i < rows ? source(i, n) : -1;
      const uint32_t dst = smem_u32(sQ) + static_cast<uint32_t>(st) * 2 * QT;
#pragma unroll 8
      for (int j = 0; j < 32; j += PER) {
        const int r = j + lane / COLS16;
        const int64_t from = __shfl_sync(0xffffffffu, at, r);
        const uint32_t to = dst + tc_at<kTcRows>(base_row + r, c);
        const int64_t src = from >= 0 ? from * D + 8 * c : 0;
        cp_async16(to, a.dout + src, from >= 0 ? 16u : 0u);
        cp_async16(to + QT, a.q + src, from >= 0 ? 16u : 0u);
      }
      cp_async_arrive(&B->q_full[st]);
    }
    cp_async_commit();
    cp_async_wait<0>();
  } else if (warp == 8) {
    // ---------------------------------------------------------------- matrix products
    {
      const uint32_t el = elect_one();
      const SmemDesc od = make_desc_sw128(smem_u32(sQ), 16, 1024), qd = make_desc_sw128(smem_u32(sQ) + QT, 16, 1024);
      const SmemDesc kd = make_desc_sw128(smem_u32(sK), 16, 1024), vd = make_desc_sw128(smem_u32(sV), 16, 1024);
      // transposed operands: 64 channels (keys) of all rows, then the next 64
      const SmemDesc ot = make_desc_sw128(smem_u32(sQ), kTcRows * 128, 1024);
      const SmemDesc qt = make_desc_sw128(smem_u32(sQ) + QT, kTcRows * 128, 1024);
      const SmemDesc pd = make_desc_sw128(smem_u32(sP), PT, 1024), gd = make_desc_sw128(smem_u32(sG), PT, 1024);
      int n_s = 0;                                  // steps whose scores are issued
      auto issue_s = [&]() {
        const int st = n_s & 1;
        if (!tc_warp_wait(&B->q_full[st], (n_s >> 1) & 1, ns)) return false;
        fence_proxy_async_smem();
        tc_fence_after();
        const uint32_t off = static_cast<uint32_t>(st * 2 * QT) >> 4;
        tc_chain<D / 16, kTcRows * 128, 32, kBaTile * 128, 32>(tmem + TM_S + st * kBaTile, SmemDesc{qd.lo + off, qd.hi},
                                                                kd, IDESC_S, 0u, el);
        tc_chain<D / 16, kTcRows * 128, 32, kBaTile * 128, 32>(tmem + TM_DP + st * kBaTile,
                                                                SmemDesc{od.lo + off, od.hi}, vd, IDESC_S, 0u, el);
        tc_commit(&B->s_full[st], el);
        ++n_s;
        return true;
      };
      for (int t = 0; t < steps; ++t) {
        const int st = t & 1;
        // Scores of step t + 1 first (their buffers were read before P(t - 1)
        // was announced), unless its rows are still on their way: step t's
        // products, which free a stage, must not wait for them.
        if (n_s == t && !issue_s()) break;
        if (t + 1 < steps && __any_sync(0xffffffffu, mbar_test(&B->q_full[st ^ 1], ((t + 1) >> 1) & 1)) && !issue_s()) break;
        if (!tc_warp_wait(&B->p_full, t & 1, ns)) break;
        tc_fence_after();
        const uint32_t off = static_cast<uint32_t>(st * 2 * QT) >> 4;
        const uint32_t more = t > 0 ? 1u : 0u;
        // K steps of 16 rows = 2048 bytes in both operands
        tc_chain<kTcRows / 16, 4 * 2048, 2048, 4 * 2048, 2048>(tmem + TM_DV, SmemDesc{ot.lo + off, ot.hi}, pd, IDESC_G,
                                                                more, el);
        if (D == 128)
          tc_chain<kTcRows / 16, 4 * 2048, 2048, 4 * 2048, 2048>(tmem + TM_DK, SmemDesc{qt.lo + off, qt.hi}, gd,
                                                                  IDESC_G, more, el);
        tc_commit(&B->q_empty[st], el);
        tc_commit(&B->p_free, el);
        if (t == steps - 1) tc_commit(&B->done, el);
      }
      tc_commit(&B->drain, el);
      mbar_wait(&B->drain, 0, 1000000000ull);
    }
  } else {
    // ---------------------------------------------------------------- P and dS
    const int grp = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t mine = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    float z_next = 0.f, d_next = 0.f;
    int seen_next = 0;
    auto row_values = [&](int t) {                  // of the next step, while this one is computed
      const int i = t * kTcRows + r;
      seen_next = 0;
      z_next = d_next = 0.f;
      if (t < steps && i < rows) {
        int n;
        const int64_t at = source(i, n);
        z_next = __ldg(a.lse_in + at);
        d_next = a.delta[at];
        seen_next = z_next != -INFINITY ? query_seen(a, len, n) : 0;   // as in the dQ kernel
      }
    };
    row_values(0);
    bool ok = true;
    for (int t = 0; t < steps; ++t) {
      const int st = t & 1;
      const float z = z_next * 1.4426950408889634f, delta = d_next;
      const int end = seen_next - key0 - 32 * grp;            // keys of this thread's 32 that the row sees
      row_values(t + 1);
      if (!tc_warp_wait(&B->s_full[st], (t >> 1) & 1, ns)) {
        ok = false;
        break;
      }
      tc_fence_after();
      float s[32], dp[32];
      tmem_ld32_sync(mine + TM_S + st * kBaTile + 32 * grp, s);
      tmem_ld32_sync(mine + TM_DP + st * kBaTile + 32 * grp, dp);
      uint32_t p[16], g[16];
      const bool part = __any_sync(0xffffffffu, end < 32);
#pragma unroll
      for (int c = 0; c < 32; c += 2) {
        float w[2], d[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          w[e] = ex2_approx(fmaf(s[c + e], a.scale_log2, -z));
          d[e] = w[e] * (dp[c + e] - delta);
          if (part) {
            w[e] = c + e < end ? w[e] : 0.f;
            d[e] = c + e < end ? d[e] : 0.f;
          }
        }
        // bf16 for the matrix products: 2^-8 relative to each
        p[c >> 1] = pack_bf16x2(w[0], w[1]);
        g[c >> 1] = pack_bf16x2(d[0], d[1]);
      }
      if (t > 0 && !tc_warp_wait(&B->p_free, (t - 1) & 1, ns)) {
        ok = false;
        break;
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t at = tc_at<kTcRows>(r, 4 * grp + c);
        *reinterpret_cast<uint4 *>(sP + at) = make_uint4(p[4 * c], p[4 * c + 1], p[4 * c + 2], p[4 * c + 3]);
        *reinterpret_cast<uint4 *>(sG + at) = make_uint4(g[4 * c], g[4 * c + 1], g[4 * c + 2], g[4 * c + 3]);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive(&B->p_full);
    }
    // ---- dV (group 0, or lanes 0-63) and dK: thread = channel, columns = keys
    if (ok && steps > 0) ok = tc_warp_wait(&B->done, 0, ns);
    tc_fence_after();
    const bool is_k = D == 128 ? grp == 1 : r >= 64;
    const int ch = D == 128 ? r : r & 63;
    const float scale = is_k ? a.scale : 1.f;
    if (D == 128 || grp == 0) {
      const uint32_t from = mine + (is_k ? TM_DK : TM_DV);
      __nv_bfloat16 *out = (is_k ? a.dk : a.dv) + (static_cast<int64_t>(head) * a.Nk + key0) * D + ch;
      float *slot = a.part_kv + (static_cast<int64_t>(a.slot_first[tile] + item - first) * 2 + !is_k) * kBaTile * D + ch;
#pragma unroll 1
      for (int c = 0; c < kBaTile; c += 32) {
        float v[32];
        if (ok && steps > 0) {
          tmem_ld32_sync(from + c, v);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          if (alone) {
            if (key0 + c + e < a.Nk) out[static_cast<int64_t>(c + e) * D] = __float2bfloat16_rn(v[e] * scale);
          } else {
            slot[(c + e) * D] = v[e] * scale;
          }
        }
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, COLS);
  }
}

}  // namespace svg
