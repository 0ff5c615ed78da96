// decode_paged_sm100.cuh -- one MALA decode step over the paged 8-bit cache
// (paged.cuh). The rule is that of decode_sm100.cuh: 128-key tiles aligned from
// position 0, newest first, the newest always kept, a later one skipped iff
// every head of the group (or the head alone) has  mt - m - ln l < ln tau -
// ln Lc.
//
// One cluster of C blocks (1 to 16) of eight warps per (sequence, key/value
// head), one launch, no workspace. A warp owns a ring of 4 KB stages (32 keys
// or values) that its lane 0 refills by TMA, so that nothing but the warp itself
// stands between a stage's use and its next load.
//
// tau > 0 (rule_kernel):
//  A  tile t goes to warp t mod 8 C: scores S[key][head] = q . k by mma
//     m16n8k16 in f16, the tile's row max m_t and mass l_t per head into the
//     block's shared memory. This reads all of K once, the HBM-bound part;
//  B  every block collects the statistics of the whole cluster and replays the
//     rule over them, newest first: all arrive at the same kept tiles, and the
//     n-th kept one falls to block n mod C;
//  C  a warp per quarter of a kept tile: P = exp(S - m) with the final m,
//     O += P V by mma; the warps' sums are joined in shared memory, the
//     blocks' through the cluster.
// tau = 0 (dense_kernel): K and V are read once, side by side; every warp keeps
// a running max, mass and output, joined at the end.
//
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
constexpr float kPShift = 14.f;      // P is carried as 2^14 p
constexpr int CK = 32;               // keys of a chunk (one ring stage)
constexpr uint32_t STAGE = CK * D;   // bytes
constexpr int MAXC = 16;             // blocks of a cluster
constexpr int RULE_NST = 3;          // ring stages of a warp
constexpr int DENSE_NST = 3;         // pairs of stages (K, V) of a warp
constexpr uint32_t RULE_RING = NW * RULE_NST * STAGE;
constexpr uint32_t DENSE_RING = NW * DENSE_NST * 2 * STAGE;

struct Params {
  Pool pool;
  const __nv_bfloat16* q;   // [batch][Hq][128]
  __nv_bfloat16* o;
  const int32_t* seq_lens;
  int G, Hkv, max_tiles;
  int C, C_log2;
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

using sm100::mbar_expect_tx;
using sm100::mbar_wait;
using sm100::smem_u32;

// Scores (raw, of the scaled q) of the sixteen keys whose rows lie at `blk` in
// the 128-byte swizzle: row r's 16-byte chunk i is at r * 128 + ((i ^ r % 8) * 16).
// Thread (r, c) takes keys r and r + 8, chunks 2 c and 2 c + 1: the eight lanes of
// a quarter-warp touch all eight chunk positions.
__device__ __forceinline__ void scores16(const unsigned char* blk, const uint32_t (&bq)[8][2],
                                         float (&acc)[4]) {
  const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  const uint32_t o0 = r * 128 + (((2 * c) ^ r) << 4), o1 = r * 128 + (((2 * c + 1) ^ r) << 4);
  uint4 a[2], b[2];
  a[0] = *reinterpret_cast<const uint4*>(blk + o0);
  a[1] = *reinterpret_cast<const uint4*>(blk + o1);
  b[0] = *reinterpret_cast<const uint4*>(blk + o0 + 1024);
  b[1] = *reinterpret_cast<const uint4*>(blk + o1 + 1024);
  const uint32_t* aw = reinterpret_cast<const uint32_t*>(a);
  const uint32_t* bw = reinterpret_cast<const uint32_t*>(b);
  acc[0] = acc[1] = acc[2] = acc[3] = 0.f;
#pragma unroll
  for (int ks = 0; ks < 8; ++ks)
    mma_f16(acc, paged::e4m3x2_to_f16x2(aw[ks]), paged::e4m3x2_to_f16x2(bw[ks]),
            paged::e4m3x2_hi_to_f16x2(aw[ks]), paged::e4m3x2_hi_to_f16x2(bw[ks]), bq[ks][0],
            bq[ks][1]);
}

// out += vs * (2^14 P) V for the sixteen values whose rows lie at `blk` (swizzled as
// above); s are their weights as packed by the score fragment's layout (keys r, r +
// 8; heads 2 c, 2 c + 1); rows from `valid` on hold nothing and count as zero
// whatever their bytes are. Rows r and r + 8 of m-block db stand for dimensions 16 r +
// 2 db and 16 r + 2 db + 1, so that a thread's sixteen bytes of a value serve all eight
// m-blocks.
__device__ __forceinline__ void add_pv16(const unsigned char* blk, int valid, const float (&w)[4],
                                         float vs, float (&out)[8][4]) {
  const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  const uint32_t b0 = movmatrix_trans(pack_f16(w[0], w[1]));
  const uint32_t b1 = movmatrix_trans(pack_f16(w[2], w[3]));
  uint4 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int key = 2 * c + (i & 1) + 8 * (i >> 1);
    v[i] = *reinterpret_cast<const uint4*>(blk + key * 128 + ((r ^ (key & 7)) << 4));
    if (key >= valid) v[i] = make_uint4(0, 0, 0, 0);
  }
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

// What the blocks of a cluster hold beside their rings.
struct Shared {
  uint64_t full[NW][3];
  uint64_t pv[NW];
  float mfin[GMAX], lfin[GMAX];  // final max (log2 units) and mass
  float wm[NW][GMAX], wl[NW][GMAX];
  int bad, abort, items;
};

// The group's place, common to both kernels.
struct Group {
  int b, h, len, nt;
  long long grp;
};

// The pages of a chunk's 32 positions: one, or two of 16 tokens. -1: none needed or
// no page of the pool (then *bad is set).
__device__ __forceinline__ void chunk_pages(const Pool& pool, int b, int pos, int len, int& id0,
                                            int& id1, int* bad) {
  id0 = id1 = -1;
  if (pos >= len) return;
  const int slot = pos >> pool.page_log2;
  id0 = paged::page_of(pool, b, slot);
  if (id0 < 0) *bad = 1;
  if (pool.page == 16 && pos + 16 < len) {
    id1 = paged::page_of(pool, b, slot + 1);
    if (id1 < 0) *bad = 1;
  }
}

// Lane 0: loads the 32 rows from position `pos` into `dst`, counted on `bar`
// (which the caller arms with chunk_bytes).
__device__ __forceinline__ void load_chunk(const CUtensorMap* map, const Pool& pool, uint32_t dst,
                                           int pos, int h, int id0, int id1, uint32_t bar) {
  if (id0 >= 0) sm100::tma_load_4d(dst, map, 0, pos & (pool.page - 1), h, id0, bar);
  if (id1 >= 0) sm100::tma_load_4d(dst + STAGE / 2, map, 0, 0, h, id1, bar);
}
__device__ __forceinline__ uint32_t chunk_bytes(const Pool& pool, int id0, int id1) {
  if (pool.page != 16) return id0 >= 0 ? STAGE : 0;
  return (id0 >= 0 ? STAGE / 2 : 0) + (id1 >= 0 ? STAGE / 2 : 0);
}

// Scores of a chunk in log2 units, -inf where there is no key (behind the
// sequence, or in a page that is not in the pool).
__device__ __forceinline__ void chunk_scores(const unsigned char* stage, const uint32_t (&bq)[8][2],
                                             int pos, int len, bool has0, bool has1, float f00,
                                             float f01, float f10, float f11, float (&s)[2][4]) {
  const int r = (threadIdx.x & 31) >> 2;
  scores16(stage, bq, s[0]);
  scores16(stage + 2048, bq, s[1]);
  s[0][0] *= f00;
  s[0][1] *= f01;
  s[0][2] *= f00;
  s[0][3] *= f01;
  s[1][0] *= f10;
  s[1][1] *= f11;
  s[1][2] *= f10;
  s[1][3] *= f11;
  if (pos + CK > len || !has0 || !has1) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool has = i ? has1 : has0;
      if (!has || pos + 16 * i + r >= len) s[i][0] = s[i][1] = kNegInf;
      if (!has || pos + 16 * i + r + 8 >= len) s[i][2] = s[i][3] = kNegInf;
    }
  }
}

// Joins the warps' and the blocks' outputs (each scaled to the same reference)
// and writes o = sum / (2^14 l).
__device__ __forceinline__ void join_and_store(const Params& p, Shared& sh, float* part,
                                               const float (&out)[8][4], const float* wscale,
                                               uint32_t rank, __nv_bfloat16* o, bool dense) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = lane >> 2, c = lane & 3;
  const int n = p.G * D;
  __syncthreads();  // the rings are free
  float* mine = part + warp * (GMAX * D);
#pragma unroll
  for (int db = 0; db < 8; ++db)
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *reinterpret_cast<float2*>(mine + (2 * c + i) * D + 16 * r + 2 * db) =
          make_float2(out[db][i] * wscale[i], out[db][2 + i] * wscale[i]);
  __syncthreads();
  for (int e = tid; e < n; e += NT) {
    float x = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) x += part[w * (GMAX * D) + e];
    part[e] = x;
  }
  const float nan = __int_as_float(0x7fc00000);
  if (p.C == 1) {
    for (int e = tid; e < n; e += NT)
      o[e] = __float2bfloat16_rn(sh.bad ? nan : part[e] / (sh.lfin[e / D] * 16384.f));
    return;
  }
  sm100::cluster_sync_all();
  const int each = (n + p.C - 1) >> p.C_log2;
  const uint32_t part_a = smem_u32(part), bad_a = smem_u32(&sh.bad), m_a = smem_u32(sh.mfin),
                 l_a = smem_u32(sh.lfin);
  for (int i = tid; i < each; i += NT) {
    const int e = (int)rank * each + i;
    if (e >= n) break;
    float x = 0.f, l = 0.f, top = kNegInf;
    int bad = 0;
    const int g = e / D;
    if (dense)
      for (int k = 0; k < p.C; ++k)
        top = fmaxf(top, sm100::ld_cluster_f32(sm100::mapa_rank(m_a + 4 * g, k)));
    for (int k = 0; k < p.C; ++k) {
      float f = 1.f;
      if (dense) {
        const float m = sm100::ld_cluster_f32(sm100::mapa_rank(m_a + 4 * g, k));
        f = m == kNegInf ? 0.f : ex2_approx(m - top);
        l += f * sm100::ld_cluster_f32(sm100::mapa_rank(l_a + 4 * g, k));
      }
      x += f * sm100::ld_cluster_f32(sm100::mapa_rank(part_a + 4 * e, k));
      bad |= (int)sm100::ld_cluster_u32(sm100::mapa_rank(bad_a, k));
    }
    if (!dense) l = sh.lfin[g];
    o[e] = __float2bfloat16_rn(bad ? nan : x / (l * 16384.f));
  }
  __syncwarp();
  sm100::cluster_sync_all();  // no block's shared memory goes while others read it
}

// An unused slot of the batch, or a length that the call did not allow for:
// the output without any work. True when there is nothing else to do.
__device__ __forceinline__ bool trivial(const Params& p, const Group& g, uint32_t rank,
                                        __nv_bfloat16* o) {
  const bool fits = g.nt <= p.max_tiles;
  if (g.nt > 0 && fits) return false;
  if (rank == 0) {
    const int tid = threadIdx.x, units = p.per_head ? p.G : 1;
    if (!fits && tid == 0) record_bad_page(0x510);
    const __nv_bfloat16 z = __float2bfloat16_rn(fits ? 0.f : __int_as_float(0x7fc00000));
    for (int e = tid; e < p.G * D; e += NT) o[e] = z;
    if (p.kept_tiles && tid < units) p.kept_tiles[g.grp * units + tid] = 0;
    if (p.keep_bits)
      for (int e = tid; e < units * p.nw; e += NT) p.keep_bits[g.grp * units * p.nw + e] = 0u;
  }
  return true;
}

__device__ __forceinline__ Group group_of(const Params& p) {
  Group g;
  g.h = blockIdx.y;
  g.b = blockIdx.z;
  g.len = p.seq_lens[g.b];
  g.nt = g.len > 0 ? (int)(((long long)g.len + T - 1) / T) : 0;
  g.grp = (long long)g.b * p.Hkv + g.h;
  return g;
}

// Statistics slots of a block: its warps' tiles, slot i * NW + warp the warp's i-th.
__host__ __device__ inline int rule_slots(int max_tiles, int C) {
  return (max_tiles + NW * C - 1) / (NW * C) * NW;
}
inline size_t rule_smem(int G, int max_tiles, int C) {
  return 1024 + RULE_RING + (size_t)rule_slots(max_tiles, C) * (G * sizeof(float2)) +
         ((size_t)(max_tiles + C - 1) / C) * sizeof(uint32_t);
}
constexpr size_t DENSE_SMEM = 1024 + DENSE_RING;

__global__ void __launch_bounds__(NT, 2) rule_kernel(const __grid_constant__ CUtensorMap tmK,
                                                     const __grid_constant__ CUtensorMap tmV,
                                                     const Params p) {
  extern __shared__ unsigned char raw[];
  __shared__ Shared sh;
  unsigned char* ring = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int c = lane & 3;
  const int G = p.G, C = p.C;
  const Pool& pool = p.pool;
  const uint32_t rank = blockIdx.x;
  const Group gr = group_of(p);
  const int len = gr.len, nt = gr.nt;
  __nv_bfloat16* o = p.o + gr.grp * G * D;
  if (trivial(p, gr, rank, o)) return;

  const int slots = rule_slots(p.max_tiles, C);
  float2* stats = reinterpret_cast<float2*>(ring + RULE_RING);               // [G][slots]
  uint32_t* list = reinterpret_cast<uint32_t*>(stats + (size_t)G * slots);   // this block's items
  if (tid == 0) {
    for (int w = 0; w < NW; ++w) {
      for (int s = 0; s < RULE_NST; ++s) sm100::mbar_init(smem_u32(&sh.full[w][s]), 1);
      sm100::mbar_init(smem_u32(&sh.pv[w]), 1);
    }
    sh.bad = sh.abort = sh.items = 0;
    sm100::fence_mbar_init();
  }
  const int units = p.per_head ? G : 1;
  if (rank == 0 && p.keep_bits)
    for (int e = tid; e < units * p.nw; e += NT) p.keep_bits[gr.grp * units * p.nw + e] = 0u;
  __syncthreads();
  volatile int* abort = &sh.abort;

  uint32_t bq[8][2];
  const float undo = load_q(p.q + gr.grp * G * D, G, bq) * p.scale_log2;
  const float undo0 = __shfl_sync(0xffffffffu, undo, 8 * c);      // head 2 c
  const float undo1 = __shfl_sync(0xffffffffu, undo, 8 * c + 4);  // head 2 c + 1

  // ---- A: statistics of this warp's tiles, a ring of chunks
  unsigned char* my = ring + warp * (RULE_NST * STAGE);
  const int W = NW * C, wg = (int)rank * NW + warp;
  const int tiles = nt > wg ? (nt - wg + W - 1) / W : 0, chunks = 4 * tiles;
  auto pos_of = [&](int k) { return (wg + (k >> 2) * W) * T + (k & 3) * CK; };
  // pages and scales of 32 chunks at a time, lane i those of the i-th; the next 32
  // are fetched while these are in use
  int id0, id1, nid0 = -1, nid1 = -1;
  float sc0 = 0.f, sc1 = 0.f, nsc0 = 0.f, nsc1 = 0.f;
  auto fetch_ids = [&](int k, int& a, int& b) {
    a = b = -1;
    if (k < chunks) chunk_pages(pool, gr.b, pos_of(k), len, a, b, &sh.bad);
  };
  auto fetch_scales = [&](int a, int b, float& x, float& y) {
    x = a >= 0 ? pool.k_scale[(long long)a * pool.Hkv + gr.h] : 0.f;
    y = b >= 0 ? pool.k_scale[(long long)b * pool.Hkv + gr.h] : x;
  };
  auto issue = [&](int k, int a, int b) {  // warp-uniform
    if (lane == 0) {
      const int s = k % RULE_NST;
      const uint32_t bar = smem_u32(&sh.full[warp][s]);
      mbar_expect_tx(bar, chunk_bytes(pool, a, b));
      load_chunk(&tmK, pool, smem_u32(my + s * STAGE), pos_of(k), gr.h, a, b, bar);
    }
  };
  fetch_ids(lane, id0, id1);
#pragma unroll
  for (int k = 0; k < RULE_NST; ++k) {
    const int a = __shfl_sync(0xffffffffu, id0, k), b = __shfl_sync(0xffffffffu, id1, k);
    if (k < chunks) issue(k, a, b);
  }
  fetch_scales(id0, id1, sc0, sc1);
  bool ok = true;
  int stage = 0;
  uint32_t phase = 0;
  for (int i = 0; i < tiles && ok; ++i) {
    if ((i & 7) == 0) {
      if (i > 0) {
        id0 = nid0;
        id1 = nid1;
        sc0 = nsc0;
        sc1 = nsc1;
      }
      fetch_ids(4 * i + 32 + lane, nid0, nid1);
    } else if ((i & 7) == 4) {
      fetch_scales(nid0, nid1, nsc0, nsc1);
    }
    float s[8][4];
#pragma unroll
    for (int qr = 0; qr < 4; ++qr) {
      const int k = 4 * i + qr, j = k & 31;
      const int a = __shfl_sync(0xffffffffu, id0, j), b = __shfl_sync(0xffffffffu, id1, j);
      const float x = __shfl_sync(0xffffffffu, sc0, j), y = __shfl_sync(0xffffffffu, sc1, j);
      ok = __all_sync(0xffffffffu,
                      ok && mbar_wait(smem_u32(&sh.full[warp][stage]), phase, abort, 0x511));
      float t2[2][4];
      chunk_scores(my + stage * STAGE, bq, pos_of(k), len, a >= 0, pool.page == 16 ? b >= 0 : a >= 0,
                   undo0 * x, undo1 * x, undo0 * y, undo1 * y, t2);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[2 * qr][e] = t2[0][e];
        s[2 * qr + 1][e] = t2[1][e];
      }
      const int nk = k + RULE_NST, nj = nk & 31;
      const bool next = (nk >> 5) != (k >> 5);
      const int na = __shfl_sync(0xffffffffu, next ? nid0 : id0, nj);
      const int nb = __shfl_sync(0xffffffffu, next ? nid1 : id1, nj);
      __syncwarp();  // every lane has read the stage
      if (nk < chunks && ok) issue(nk, na, nb);
      if (++stage == RULE_NST) {
        stage = 0;
        phase ^= 1;
      }
    }
    float m0 = kNegInf, m1 = kNegInf;
#pragma unroll
    for (int kb = 0; kb < 8; ++kb) {
      m0 = fmaxf(m0, fmaxf(s[kb][0], s[kb][2]));
      m1 = fmaxf(m1, fmaxf(s[kb][1], s[kb][3]));
    }
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) {
      m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, x));
      m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, x));
    }
    // a tile without a finite score: mass 0
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
      if (2 * c < G) stats[2 * c * slots + i * NW + warp] = make_float2(m0, l0);
      if (2 * c + 1 < G) stats[(2 * c + 1) * slots + i * NW + warp] = make_float2(m1, l1);
    }
  }
  if (!ok) sm100::drain_in_flight();
  __syncwarp();
  if (C > 1)
    sm100::cluster_sync_all();
  else
    __syncthreads();

  // ---- B: the rule over all tiles, newest first, in stretches that fit in the
  // ring's space (a single block's statistics lie in tile order already)
  {
    float2* loc = C > 1 ? reinterpret_cast<float2*>(ring) : stats;
    const int cap = C > 1 ? ((int)(RULE_RING / sizeof(float2)) / G) & ~31 : slots;
    const uint32_t stats_a = smem_u32(stats);
    const float thr = p.log2_tau - lg2_approx((float)len);
    const uint32_t all = (1u << G) - 1u;
    float m[GMAX], l[GMAX], bound[GMAX];
    int cnt[GMAX];
    int count = 0, next = nt - 1;
#pragma unroll
    for (int g = 0; g < GMAX; ++g) {
      m[g] = kNegInf;
      l[g] = 0.f;
      cnt[g] = 0;
      bound[g] = kNegInf;
    }
    for (int hi = nt; hi > 0;) {
      const int lo = C > 1 ? max(0, hi - cap) : 0;
      if (C > 1) {
        const int n = hi - lo;
        for (int g = 0; g < G; ++g)
          for (int e = tid; e < n; e += NT) {
            const int t = lo + e, w = t & (W - 1);
            const uint32_t at = stats_a + 8u * (uint32_t)(g * slots + (t / W) * NW + (w & (NW - 1)));
            loc[g * cap + e] = sm100::ld_cluster_f32x2(sm100::mapa_rank(at, w / NW));
          }
        __syncthreads();
      }
      if (warp == 0) {
        auto take = [&](int t, uint32_t hm) {
#pragma unroll
          for (int g = 0; g < GMAX; ++g) {
            if (!((hm >> g) & 1u)) continue;
            const float2 s = loc[g * cap + t - lo];
            const float mn = fmaxf(m[g], s.x);
            const float z = mn == kNegInf ? 0.f : mn;
            l[g] = l[g] * ex2_approx(m[g] - z) + s.y * ex2_approx(s.x - z);
            m[g] = mn;
            bound[g] = mn + lg2_approx(l[g]) + thr;
            ++cnt[g];
            if (p.keep_bits && rank == 0 && lane == 0 && (p.per_head || g == 0))
              p.keep_bits[(gr.grp * units + (p.per_head ? g : 0)) * p.nw + (t >> 5)] |= 1u << (t & 31);
          }
          if (lane == 0 && (count & (C - 1)) == (int)rank) list[count >> p.C_log2] = (uint32_t)t | hm << 24;
          ++count;
        };
        if (next == nt - 1) {
          take(next, all);
          --next;
        }
        while (next >= lo) {
          const int t = next - lane;
          uint32_t want = 0;
          if (t >= lo) {
#pragma unroll
            for (int g = 0; g < GMAX; ++g)  // a NaN keeps
              if (g < G && !(loc[g * cap + t - lo].x < bound[g])) want |= 1u << g;
            if (!p.per_head && want) want = all;
          }
          const unsigned vote = __ballot_sync(0xffffffffu, want != 0u);
          if (!vote) {
            next -= 32;
            continue;
          }
          const int src = __ffs(vote) - 1;
          take(next - src, __shfl_sync(0xffffffffu, want, src));
          next -= src + 1;
        }
        next = lo - 1;
      }
      hi = lo;
      if (hi > 0) __syncthreads();
    }
    if (warp == 0) {
      if (lane == 0) sh.items = (count - (int)rank + C - 1) >> p.C_log2;
#pragma unroll
      for (int g = 0; g < GMAX; ++g)
        if (lane == g) {
          sh.mfin[g] = m[g] == kNegInf ? 0.f : m[g];
          sh.lfin[g] = l[g];
          if (p.kept_tiles && rank == 0 && g < units) p.kept_tiles[gr.grp * units + g] = cnt[g];
        }
    }
    sm100::fence_proxy_async_smem();  // the ring's space goes back to the TMA
    __syncthreads();
  }

  // ---- C: values of this block's kept tiles, a warp per chunk
  float out[8][4];
#pragma unroll
  for (int db = 0; db < 8; ++db)
#pragma unroll
    for (int i = 0; i < 4; ++i) out[db][i] = 0.f;
  const float m0 = sh.mfin[2 * c], m1 = sh.mfin[2 * c + 1];
  const int n_chunks = sh.items * 4;
  phase = 0;
  for (int x = warp; x < n_chunks && ok; x += NW) {
    const uint32_t ent = list[x >> 2];
    const int pos = (int)(ent & 0xffffffu) * T + (x & 3) * CK;
    if (pos >= len) continue;
    int a, b;
    chunk_pages(pool, gr.b, pos, len, a, b, &sh.bad);
    const uint32_t bar = smem_u32(&sh.pv[warp]);
    __syncwarp();
    if (lane == 0) {
      mbar_expect_tx(bar, 2 * chunk_bytes(pool, a, b));
      load_chunk(&tmK, pool, smem_u32(my), pos, gr.h, a, b, bar);
      load_chunk(&tmV, pool, smem_u32(my + STAGE), pos, gr.h, a, b, bar);
    }
    float x0, x1, v0, v1;
    fetch_scales(a, b, x0, x1);
    v0 = a >= 0 ? pool.v_scale[(long long)a * pool.Hkv + gr.h] : 0.f;
    v1 = b >= 0 ? pool.v_scale[(long long)b * pool.Hkv + gr.h] : v0;
    ok = __all_sync(0xffffffffu, mbar_wait(bar, phase, abort, 0x512));
    phase ^= 1;
    const bool has1 = pool.page == 16 ? b >= 0 : a >= 0;
    float s[2][4];
    chunk_scores(my, bq, pos, len, a >= 0, has1, undo0 * x0, undo1 * x0, undo0 * x1, undo1 * x1, s);
    const bool on0 = (ent >> (24 + 2 * c)) & 1u, on1 = (2 * c + 1 < 8) && (ent >> (25 + 2 * c)) & 1u;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float w[4];
      w[0] = on0 ? ex2_approx(s[i][0] - m0 + kPShift) : 0.f;
      w[1] = on1 ? ex2_approx(s[i][1] - m1 + kPShift) : 0.f;
      w[2] = on0 ? ex2_approx(s[i][2] - m0 + kPShift) : 0.f;
      w[3] = on1 ? ex2_approx(s[i][3] - m1 + kPShift) : 0.f;
      if (i ? has1 : a >= 0) add_pv16(my + STAGE + i * 2048, len - pos - 16 * i, w, i ? v1 : v0, out);
    }
  }
  if (!ok) sm100::drain_in_flight();
  __syncwarp();
  const float one[2] = {1.f, 1.f};
  join_and_store(p, sh, reinterpret_cast<float*>(ring), out, one, rank, o, false);
}

__global__ void __launch_bounds__(NT, 1) dense_kernel(const __grid_constant__ CUtensorMap tmK,
                                                      const __grid_constant__ CUtensorMap tmV,
                                                      const Params p) {
  extern __shared__ unsigned char raw[];
  __shared__ Shared sh;
  unsigned char* ring = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int c = lane & 3;
  const int G = p.G, C = p.C;
  const Pool& pool = p.pool;
  const uint32_t rank = blockIdx.x;
  const Group gr = group_of(p);
  const int len = gr.len, nt = gr.nt;
  __nv_bfloat16* o = p.o + gr.grp * G * D;
  if (trivial(p, gr, rank, o)) return;
  if (tid == 0) {
    for (int w = 0; w < NW; ++w)
      for (int s = 0; s < DENSE_NST; ++s) sm100::mbar_init(smem_u32(&sh.full[w][s]), 1);
    sh.bad = sh.abort = 0;
    sm100::fence_mbar_init();
  }
  const int units = p.per_head ? G : 1;
  if (rank == 0) {  // every tile is kept
    if (p.kept_tiles && tid < units) p.kept_tiles[gr.grp * units + tid] = nt;
    if (p.keep_bits)
      for (int e = tid; e < units * p.nw; e += NT) {
        const int left = nt - 32 * (e % p.nw);
        p.keep_bits[gr.grp * units * p.nw + e] =
            left >= 32 ? 0xffffffffu : (left > 0 ? (1u << left) - 1u : 0u);
      }
  }
  __syncthreads();
  volatile int* abort = &sh.abort;

  uint32_t bq[8][2];
  const float undo = load_q(p.q + gr.grp * G * D, G, bq) * p.scale_log2;
  const float undo0 = __shfl_sync(0xffffffffu, undo, 8 * c);
  const float undo1 = __shfl_sync(0xffffffffu, undo, 8 * c + 4);

  unsigned char* my = ring + warp * (DENSE_NST * 2 * STAGE);
  const int W = NW * C, wg = (int)rank * NW + warp;
  const int all = (int)(((long long)len + CK - 1) / CK);
  const int chunks = all > wg ? (all - wg + W - 1) / W : 0;
  auto pos_of = [&](int k) { return (wg + k * W) * CK; };
  int id0, id1, nid0 = -1, nid1 = -1;
  float4 sc = make_float4(0.f, 0.f, 0.f, 0.f), nsc = sc;  // k, k (second page), v, v
  auto fetch_ids = [&](int k, int& a, int& b) {
    a = b = -1;
    if (k < chunks) chunk_pages(pool, gr.b, pos_of(k), len, a, b, &sh.bad);
  };
  auto fetch_scales = [&](int a, int b, float4& x) {
    x.x = a >= 0 ? pool.k_scale[(long long)a * pool.Hkv + gr.h] : 0.f;
    x.z = a >= 0 ? pool.v_scale[(long long)a * pool.Hkv + gr.h] : 0.f;
    x.y = b >= 0 ? pool.k_scale[(long long)b * pool.Hkv + gr.h] : x.x;
    x.w = b >= 0 ? pool.v_scale[(long long)b * pool.Hkv + gr.h] : x.z;
  };
  auto issue = [&](int k, int a, int b) {
    if (lane == 0) {
      const int s = k % DENSE_NST;
      const uint32_t bar = smem_u32(&sh.full[warp][s]), dst = smem_u32(my + s * 2 * STAGE);
      mbar_expect_tx(bar, 2 * chunk_bytes(pool, a, b));
      load_chunk(&tmK, pool, dst, pos_of(k), gr.h, a, b, bar);
      load_chunk(&tmV, pool, dst + STAGE, pos_of(k), gr.h, a, b, bar);
    }
  };
  fetch_ids(lane, id0, id1);
#pragma unroll
  for (int k = 0; k < DENSE_NST; ++k) {
    const int a = __shfl_sync(0xffffffffu, id0, k), b = __shfl_sync(0xffffffffu, id1, k);
    if (k < chunks) issue(k, a, b);
  }
  fetch_scales(id0, id1, sc);

  float out[8][4];
#pragma unroll
  for (int db = 0; db < 8; ++db)
#pragma unroll
    for (int i = 0; i < 4; ++i) out[db][i] = 0.f;
  float m0 = kNegInf, m1 = kNegInf, l0 = 0.f, l1 = 0.f;  // l: this lane's keys only
  bool ok = true;
  int stage = 0;
  uint32_t phase = 0;
  for (int k = 0; k < chunks && ok; ++k) {
    const int j = k & 31;
    if (j == 0) {
      if (k > 0) {
        id0 = nid0;
        id1 = nid1;
        sc = nsc;
      }
      fetch_ids(k + 32 + lane, nid0, nid1);
    } else if (j == 16) {
      fetch_scales(nid0, nid1, nsc);
    }
    const int a = __shfl_sync(0xffffffffu, id0, j), b = __shfl_sync(0xffffffffu, id1, j);
    const float x0 = __shfl_sync(0xffffffffu, sc.x, j), x1 = __shfl_sync(0xffffffffu, sc.y, j);
    const float v0 = __shfl_sync(0xffffffffu, sc.z, j), v1 = __shfl_sync(0xffffffffu, sc.w, j);
    const bool has1 = pool.page == 16 ? b >= 0 : a >= 0;
    const int pos = pos_of(k);
    ok = __all_sync(0xffffffffu,
                    mbar_wait(smem_u32(&sh.full[warp][stage]), phase, abort, 0x513));
    const unsigned char* st = my + stage * 2 * STAGE;
    float s[2][4];
    chunk_scores(st, bq, pos, len, a >= 0, has1, undo0 * x0, undo1 * x0, undo0 * x1, undo1 * x1, s);
    float t0 = fmaxf(fmaxf(s[0][0], s[0][2]), fmaxf(s[1][0], s[1][2]));
    float t1 = fmaxf(fmaxf(s[0][1], s[0][3]), fmaxf(s[1][1], s[1][3]));
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) {
      t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, x));
      t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, x));
    }
    if (__any_sync(0xffffffffu, t0 > m0 || t1 > m1)) {
      const float n0 = fmaxf(m0, t0), n1 = fmaxf(m1, t1);
      const float f0 = m0 == kNegInf ? 0.f : ex2_approx(m0 - n0);
      const float f1 = m1 == kNegInf ? 0.f : ex2_approx(m1 - n1);
      m0 = n0;
      m1 = n1;
      l0 *= f0;
      l1 *= f1;
#pragma unroll
      for (int db = 0; db < 8; ++db) {
        out[db][0] *= f0;
        out[db][2] *= f0;
        out[db][1] *= f1;
        out[db][3] *= f1;
      }
    }
    const float z0 = m0 == kNegInf ? 0.f : m0 - kPShift, z1 = m1 == kNegInf ? 0.f : m1 - kPShift;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float w[4];
      w[0] = ex2_approx(s[i][0] - z0);
      w[1] = ex2_approx(s[i][1] - z1);
      w[2] = ex2_approx(s[i][2] - z0);
      w[3] = ex2_approx(s[i][3] - z1);
      l0 += w[0] + w[2];
      l1 += w[1] + w[3];
      if (i ? has1 : a >= 0) add_pv16(st + STAGE + i * 2048, len - pos - 16 * i, w, i ? v1 : v0, out);
    }
    const int nk = k + DENSE_NST, nj = nk & 31;
    const bool next = (nk >> 5) != (k >> 5);
    const int na = __shfl_sync(0xffffffffu, next ? nid0 : id0, nj);
    const int nb = __shfl_sync(0xffffffffu, next ? nid1 : id1, nj);
    __syncwarp();  // every lane has read the stages
    if (nk < chunks && ok) issue(nk, na, nb);
    if (++stage == DENSE_NST) {
      stage = 0;
      phase ^= 1;
    }
  }
  if (!ok) sm100::drain_in_flight();
#pragma unroll
  for (int x = 4; x < 32; x <<= 1) {
    l0 += __shfl_xor_sync(0xffffffffu, l0, x);
    l1 += __shfl_xor_sync(0xffffffffu, l1, x);
  }
  if (lane < 4) {
    sh.wm[warp][2 * c] = m0;
    sh.wm[warp][2 * c + 1] = m1;
    sh.wl[warp][2 * c] = l0;
    sh.wl[warp][2 * c + 1] = l1;
  }
  __syncthreads();
  float top0 = kNegInf, top1 = kNegInf;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    top0 = fmaxf(top0, sh.wm[w][2 * c]);
    top1 = fmaxf(top1, sh.wm[w][2 * c + 1]);
  }
  if (tid < GMAX) {
    float top = kNegInf, sum = 0.f;
    for (int w = 0; w < NW; ++w) top = fmaxf(top, sh.wm[w][tid]);
    for (int w = 0; w < NW; ++w) {
      const float x = sh.wm[w][tid];
      sum += x == kNegInf ? sh.wl[w][tid] * 0.f : sh.wl[w][tid] * ex2_approx(x - top);
    }
    sh.mfin[tid] = top;
    sh.lfin[tid] = sum * (1.f / 16384.f);
  }
  const float scale[2] = {m0 == kNegInf ? 0.f : ex2_approx(m0 - top0),
                          m1 == kNegInf ? 0.f : ex2_approx(m1 - top1)};
  join_and_store(p, sh, reinterpret_cast<float*>(ring), out, scale, rank, o, true);
}

}  // namespace pdec
}  // namespace mala
