// decode_paged_sm100.cuh -- one MALA decode step over the paged 8-bit cache
// (paged.cuh). The rule is that of decode_sm100.cuh: 128-key tiles aligned from
// position 0, newest first, the newest always kept, a later one skipped iff
// every head of the group (or the head alone) has  mt - m - ln l < ln tau -
// ln Lc.
//
// One block of eight warps per (sequence, key/value head):
//  A  a warp per tile: scores S[key][head] = q . k by mma m16n8k16 in f16,
//     the tile's row max m_t and mass l_t per head into shared memory;
//  B  one warp replays the rule over (m_t, l_t);
//  C  a warp per quarter of a kept tile: P = exp(S - m), O += P V by mma;
//     the warps' sums are joined in shared memory.
// The number formats: e4m3 is exact in f16; q is scaled by a power of two per
// head so that its largest value is in [2^14, 2^15), where all values within
// 2^-29 of the largest are exact in f16 and smaller ones are off by at most 2^-39
// of it, less than a float32 sum's rounding; P is carried as 2^14 p, which keeps
// eleven bits down to p = 2^-28. Sums are float32.
#pragma once

#include "paged.cuh"
#include "sm100.cuh"

namespace mala {
namespace pdec {

using paged::D;
using paged::Pool;
using sm100::ex2_approx;

constexpr int T = 128;
constexpr int GMAX = 8;
constexpr int NW = 8;
constexpr int NT = NW * 32;
constexpr float kPShift = 14.f;

struct Params {
  Pool pool;
  const __nv_bfloat16* q;   // [batch][Hq][128]
  __nv_bfloat16* o;
  const int32_t* seq_lens;
  int G, Hkv, max_tiles;
  float scale_log2, log2_tau;
  int never_skip, per_head;
  int32_t* kept_tiles;
  uint32_t* keep_bits;
  int nw;  // words of a keep_bits row
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float lg2_approx(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// B fragments of the group's heads for S = K q^T. The order of a sum's terms
// is free, so thread c = lane % 4 takes dimensions 32 c .. 32 c + 31 (the bytes
// it loads of a key) instead of the fragment's own columns: k-step ks covers
// dimensions 32 c + 4 ks .. + 3. Returns the factor that undoes head n =
// lane / 4's scaling.
__device__ __forceinline__ float load_q(const __nv_bfloat16* q, int G, uint32_t (&bq)[8][2]) {
  const int lane = threadIdx.x & 31, n = lane >> 2, c = lane & 3;
  float x[32];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint4 u = make_uint4(0, 0, 0, 0);
    if (n < G) u = *reinterpret_cast<const uint4*>(q + n * D + 32 * c + 8 * i);
    float y[8];
    paged::unpack8(u, y);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[8 * i + e] = y[e];
      amax = fmaxf(amax, fabsf(y[e]));
    }
  }
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  int e = (int)(__float_as_uint(amax) >> 23);  // biased exponent
  e = e < 30 ? 30 : (e > 240 ? 240 : e);
  const float up = __uint_as_float((uint32_t)(127 + 14 - (e - 127)) << 23);
#pragma unroll
  for (int ks = 0; ks < 8; ++ks) {
    bq[ks][0] = pack_f16(x[4 * ks] * up, x[4 * ks + 1] * up);
    bq[ks][1] = pack_f16(x[4 * ks + 2] * up, x[4 * ks + 3] * up);
  }
  return __uint_as_float((uint32_t)(127 - 14 + (e - 127)) << 23);
}

// Scores (raw, of the scaled q) of sixteen keys; `row` is key lane / 4's
// address, `row8` that of the key eight further on.
__device__ __forceinline__ void scores16(const uint8_t* row, const uint8_t* row8,
                                         const uint32_t (&bq)[8][2], float (&acc)[4]) {
  const int c = threadIdx.x & 3;
  uint4 a[2], b[2];
  a[0] = *reinterpret_cast<const uint4*>(row + 32 * c);
  a[1] = *reinterpret_cast<const uint4*>(row + 32 * c + 16);
  b[0] = *reinterpret_cast<const uint4*>(row8 + 32 * c);
  b[1] = *reinterpret_cast<const uint4*>(row8 + 32 * c + 16);
  const uint32_t* aw = reinterpret_cast<const uint32_t*>(a);
  const uint32_t* bw = reinterpret_cast<const uint32_t*>(b);
  acc[0] = acc[1] = acc[2] = acc[3] = 0.f;
#pragma unroll
  for (int ks = 0; ks < 8; ++ks)
    mma_f16(acc, paged::e4m3x2_to_f16x2(aw[ks]), paged::e4m3x2_to_f16x2(bw[ks]),
            paged::e4m3x2_hi_to_f16x2(aw[ks]), paged::e4m3x2_hi_to_f16x2(bw[ks]), bq[ks][0],
            bq[ks][1]);
}

struct Smem {
  float mfin[GMAX], lfin[GMAX];
  int count, bad;
};

__global__ void __launch_bounds__(NT) decode_kernel(const Params p) {
  extern __shared__ __align__(16) unsigned char raw[];
  __shared__ Smem sh;
  // [G][max_tiles] statistics, then kept tiles and heads; the partial outputs
  // reuse the space
  float2* stats = reinterpret_cast<float2*>(raw);
  int* kept = reinterpret_cast<int*>(stats + p.G * p.max_tiles);
  uint8_t* heads = reinterpret_cast<uint8_t*>(kept + p.max_tiles);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.x, b = blockIdx.y, G = p.G;
  const int r = lane >> 2, c = lane & 3;
  const Pool& pool = p.pool;
  const int len = p.seq_lens[b];
  const int nt = len > 0 ? (int)(((long long)len + T - 1) / T) : 0;
  const bool fits = nt <= p.max_tiles;
  __nv_bfloat16* o = p.o + ((long long)b * p.Hkv + h) * G * D;
  const long long grp = (long long)b * p.Hkv + h;
  if (tid == 0) sh.bad = 0;
  if (p.keep_bits) {
    const int n = (p.per_head ? G : 1) * p.nw;
    for (int e = tid; e < n; e += NT) p.keep_bits[grp * n + e] = 0u;
  }
  if (nt == 0 || !fits) {  // an unused slot, or a length that the call did not allow for
    if (!fits && tid == 0) record_bad_page(0x510);
    const __nv_bfloat16 z = __float2bfloat16_rn(fits ? 0.f : __int_as_float(0x7fc00000));
    for (int e = tid; e < G * D; e += NT) o[e] = z;
    if (p.kept_tiles && tid < (p.per_head ? G : 1)) p.kept_tiles[grp * (p.per_head ? G : 1) + tid] = 0;
    return;
  }
  __syncthreads();

  uint32_t bq[8][2];
  const float undo = load_q(p.q + grp * G * D, G, bq) * p.scale_log2;
  const float undo0 = __shfl_sync(0xffffffffu, undo, 8 * c);      // head 2 c
  const float undo1 = __shfl_sync(0xffffffffu, undo, 8 * c + 4);  // head 2 c + 1

  // scores of sixteen keys from position pos0, in log2 units; -inf where no key is
  auto scores = [&](int pos0, float (&s)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = kNegInf;
    if (pos0 >= len) return;
    const int id = paged::page_of(pool, b, pos0 / pool.page);
    if (id < 0) {
      sh.bad = 1;
      return;
    }
    const uint8_t* base = pool.k + id * pool.k_page + h * pool.k_head +
                          (pos0 % pool.page) * pool.k_tok;
    float acc[4];
    scores16(base + r * pool.k_tok, base + (r + 8) * pool.k_tok, bq, acc);
    const float ks = pool.k_scale[(long long)id * pool.Hkv + h];
    if (pos0 + r < len) {
      s[0] = acc[0] * (undo0 * ks);
      s[1] = acc[1] * (undo1 * ks);
    }
    if (pos0 + r + 8 < len) {
      s[2] = acc[2] * (undo0 * ks);
      s[3] = acc[3] * (undo1 * ks);
    }
  };

  // A: statistics
  for (int t = warp; t < nt; t += NW) {
    float s[8][4];
    float m0 = kNegInf, m1 = kNegInf;
#pragma unroll
    for (int kb = 0; kb < 8; ++kb) {
      scores(t * T + kb * 16, s[kb]);
      m0 = fmaxf(m0, fmaxf(s[kb][0], s[kb][2]));
      m1 = fmaxf(m1, fmaxf(s[kb][1], s[kb][3]));
    }
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) {
      m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, x));
      m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, x));
    }
    // a tile of -inf scores only (a key's scale or q beyond float32): mass 0
    const float z0 = m0 == kNegInf ? 0.f : m0, z1 = m1 == kNegInf ? 0.f : m1;
    float l0 = 0.f, l1 = 0.f;
#pragma unroll
    for (int kb = 0; kb < 8; ++kb) {
      l0 += ex2_approx(s[kb][0] - z0) + ex2_approx(s[kb][2] - z0);
      l1 += ex2_approx(s[kb][1] - z1) + ex2_approx(s[kb][3] - z1);
    }
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, x);
      l1 += __shfl_xor_sync(0xffffffffu, l1, x);
    }
    if (isnan(l0)) m0 = l0;  // a tile with a NaN score is kept, and shows
    if (isnan(l1)) m1 = l1;
    if (lane < 4) {
      if (2 * c < G) stats[2 * c * p.max_tiles + t] = make_float2(m0, l0);
      if (2 * c + 1 < G) stats[(2 * c + 1) * p.max_tiles + t] = make_float2(m1, l1);
    }
  }
  __syncthreads();

  // B: the rule, newest first
  if (warp == 0) {
    const float thr = p.never_skip ? kNegInf : p.log2_tau - lg2_approx((float)len);
    const uint32_t all = (1u << G) - 1u;
    float m[GMAX], l[GMAX], bound[GMAX];
    int cnt[GMAX];
    int count = 0;
#pragma unroll
    for (int g = 0; g < GMAX; ++g) {
      m[g] = kNegInf;
      l[g] = 0.f;
      cnt[g] = 0;
      bound[g] = kNegInf;
    }
    auto take = [&](int t, uint32_t hm) {
#pragma unroll
      for (int g = 0; g < GMAX; ++g) {
        if (!((hm >> g) & 1u)) continue;
        const float2 s = stats[g * p.max_tiles + t];
        const float mn = fmaxf(m[g], s.x);
        const float z = mn == kNegInf ? 0.f : mn;
        l[g] = l[g] * ex2_approx(m[g] - z) + s.y * ex2_approx(s.x - z);
        m[g] = mn;
        bound[g] = mn + lg2_approx(l[g]) + thr;
        ++cnt[g];
        if (p.keep_bits && lane == 0 && (p.per_head || g == 0))
          p.keep_bits[(p.per_head ? grp * G + g : grp) * p.nw + (t >> 5)] |= 1u << (t & 31);
      }
      if (lane == 0) {
        kept[count] = t;
        heads[count] = (uint8_t)hm;
      }
      ++count;
    };
    take(nt - 1, all);
    int next = nt - 2;
    while (next >= 0) {
      const int t = next - lane;
      uint32_t want = 0;
      if (t >= 0) {
#pragma unroll
        for (int g = 0; g < GMAX; ++g)  // NaN keeps
          if (g < G && (p.never_skip || !(stats[g * p.max_tiles + t].x < bound[g])))
            want |= 1u << g;
        if (!p.per_head && want) want = all;
      }
      const unsigned vote = __ballot_sync(0xffffffffu, want != 0u);
      if (!vote) {
        next -= 32;
        continue;
      }
      const int src = __ffs(vote) - 1;
      take(next - src, __shfl_sync(0xffffffffu, want, src));
      __syncwarp();
      next -= src + 1;
    }
    if (lane == 0) sh.count = count;
#pragma unroll
    for (int g = 0; g < GMAX; ++g)
      if (lane == g) {
        sh.mfin[g] = m[g] == kNegInf ? 0.f : m[g];
        sh.lfin[g] = l[g];
        if (p.kept_tiles) {
          if (p.per_head && g < G) p.kept_tiles[grp * G + g] = cnt[g];
          if (!p.per_head && g == 0) p.kept_tiles[grp] = cnt[0];
        }
      }
  }
  __syncthreads();

  // C: values. Rows r and r + 8 of m-block db stand for dimensions 16 r + 2 db
  // and 16 r + 2 db + 1, so that a thread's sixteen bytes of a key serve all
  // eight m-blocks.
  float out[8][4];
#pragma unroll
  for (int db = 0; db < 8; ++db)
#pragma unroll
    for (int i = 0; i < 4; ++i) out[db][i] = 0.f;
  const float m0 = sh.mfin[2 * c], m1 = sh.mfin[2 * c + 1];
  for (int item = warp; item < sh.count * 8; item += NW) {
    const int pos0 = kept[item >> 3] * T + (item & 7) * 16;
    if (pos0 >= len) continue;
    const uint32_t hm = heads[item >> 3];
    float s[4];
    scores(pos0, s);
    const int id = paged::page_of(pool, b, pos0 / pool.page);
    if (id < 0) continue;
    const bool on0 = (hm >> (2 * c)) & 1u, on1 = (hm >> (2 * c + 1)) & 1u;
    const float p0 = on0 ? ex2_approx(s[0] - m0 + kPShift) : 0.f;
    const float p1 = on1 ? ex2_approx(s[1] - m1 + kPShift) : 0.f;
    const float p2 = on0 ? ex2_approx(s[2] - m0 + kPShift) : 0.f;
    const float p3 = on1 ? ex2_approx(s[3] - m1 + kPShift) : 0.f;
    const uint32_t b0 = movmatrix_trans(pack_f16(p0, p1));
    const uint32_t b1 = movmatrix_trans(pack_f16(p2, p3));
    const uint8_t* base = pool.v + id * pool.v_page + h * pool.v_head +
                          (pos0 % pool.page) * pool.v_tok;
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int key = 2 * c + (i & 1) + 8 * (i >> 1);
      v[i] = make_uint4(0, 0, 0, 0);
      if (pos0 + key < len)
        v[i] = *reinterpret_cast<const uint4*>(base + key * pool.v_tok + 16 * r);
    }
    const float vs = pool.v_scale[(long long)id * pool.Hkv + h];
    const uint32_t* w0 = reinterpret_cast<const uint32_t*>(&v[0]);
    const uint32_t* w1 = reinterpret_cast<const uint32_t*>(&v[1]);
    const uint32_t* w2 = reinterpret_cast<const uint32_t*>(&v[2]);
    const uint32_t* w3 = reinterpret_cast<const uint32_t*>(&v[3]);
#pragma unroll
    for (int db = 0; db < 8; ++db) {
      const uint32_t sel = (db & 1) ? 0x7362 : 0x5140;
      const uint32_t lo = __byte_perm(w0[db >> 1], w1[db >> 1], sel);
      const uint32_t hi = __byte_perm(w2[db >> 1], w3[db >> 1], sel);
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
      mma_f16(acc, paged::e4m3x2_to_f16x2(lo), paged::e4m3x2_hi_to_f16x2(lo),
              paged::e4m3x2_to_f16x2(hi), paged::e4m3x2_hi_to_f16x2(hi), b0, b1);
#pragma unroll
      for (int i = 0; i < 4; ++i) out[db][i] = fmaf(acc[i], vs, out[db][i]);
    }
  }
  __syncthreads();
  float* part = reinterpret_cast<float*>(raw);  // [GMAX][128], joined warp by warp
  for (int w = 0; w < NW; ++w) {
    if (warp == w) {
#pragma unroll
      for (int db = 0; db < 8; ++db)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float* at = part + (2 * c + (i & 1)) * D + 16 * r + 2 * db + (i >> 1);
          *at = (w ? *at : 0.f) + out[db][i];
        }
    }
    __syncthreads();
  }
  const bool bad = sh.bad != 0;
  for (int e = tid; e < G * D; e += NT) {
    const float l = sh.lfin[e / D] * 16384.f;
    o[e] = __float2bfloat16_rn(bad ? __int_as_float(0x7fc00000) : part[e] / l);
  }
}

// Statistics, the list of kept tiles and its heads; at least the joined output.
inline size_t smem_bytes(int G, int max_tiles) {
  const size_t n = (size_t)max_tiles * (G * sizeof(float2) + 5);
  const size_t out = GMAX * D * sizeof(float);
  return ((n > out ? n : out) + 15) & ~size_t(15);
}

}  // namespace pdec
}  // namespace mala
