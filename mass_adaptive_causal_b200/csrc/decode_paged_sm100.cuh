// decode_paged_sm100.cuh -- one MALA decode step over the paged 8-bit cache
// (paged.cuh). The rule is that of decode_sm100.cuh: 128-key tiles aligned from
// position 0, newest first, the newest always kept, a later one skipped iff
// every head of the group (or the head alone) has  mt - m - ln l < ln tau -
// ln Lc.
//
// One cluster of C blocks (1 to 16) per (sequence, key/value head), one launch, no
// workspace; tile t of the sequence is block t mod C's. A block has four warps that do the
// softmax (a thread per key of a tile, later per dimension of the output), two that look
// pages up and load tiles by TMA into a ring, and one that issues the matrix products.
//
// tau > 0 (RULE):
//  A  scores of every tile, its max m_t and mass l_t per head into the block's shared
//     memory. This reads all of K once, the HBM-bound part;
//  B  every block collects the statistics of the whole cluster and replays the
//     rule over them, newest first: all arrive at the same kept tiles, and the
//     n-th kept one falls to block n mod C;
//  C  for its kept tiles: P = exp(S - m), O += P V; the blocks' sums are joined through the
//     cluster.
// tau = 0: K and V are read once, side by side, with a running max, mass and output.
//
// Both products run on tcgen05 in e4m3, straight on the bytes as they lie in the cache:
// S[key][.] = K q^T with the K tile as the 128-row operand, O[dim][.] = V^T P with the
// V tile as the (transposed) 128-row operand. (mma.sync has no e4m3 form of its own here: it
// is widened to f16, which made a warp's integer work the bound at 45% of the copy
// bandwidth.) The other operand is split into four e4m3 terms, 2^4 apart, in columns of their
// own, and the columns' sums are joined in float32:
//  - q, scaled by a power of two per head to have its largest value in [2^7, 2^8): a bf16
//    value has eight bits, a term carries four, so values within 2^-21 of the largest are
//    exact, and the rest is off by at most 2^-29 of it;
//  - P, scaled to 2^8 at the row's reference (its running or final max), is split from float32,
//    what its first term leaves going on in f16: off by at most 2^-16 of itself, or 2^-30 of
//    the reference.
// The kernel is bound by HBM: 16 x 131072 tokens of 8 heads, tau = 1: 326 us (2.15 GB of K, the
// measured copy bandwidth); 16 x 8192, tau = 0: 47 us (5.7 TB/s, 87%); short caches by latency:
// 1 x 1000: 8.7 us. Two blocks to an SM: while one waits at its ends, the other streams.
// Sums are float32; a row's max and mass never leave float32.
#pragma once

#include "paged.cuh"
#include "sm100.cuh"

namespace mala {
namespace pdec {

using paged::D;
using paged::Pool;
using sm100::ex2_approx;
using sm100::mbar_arrive;
using sm100::mbar_expect_tx;
using sm100::mbar_wait;
using sm100::smem_u32;

constexpr int T = 128;
constexpr int GMAX = 8;
constexpr int NT = 256;               // warps 0 - 3 softmax, 4 and 7 load, 5 products, 6 holds the
                                      // tensor memory
constexpr int NC = 128;               // softmax threads
static_assert(NT - 64 == 192, "the number in the second named barrier");
constexpr int W_MMA = 5, W_TMEM = 6;
constexpr int W_LOAD = 4, W_LOAD2 = 7;  // even and odd tiles: one warp's loop bounded a block's rate
constexpr uint32_t TILE_BYTES = T * D;
constexpr int NST = 5;                // ring stages (tiles)
constexpr uint32_t RING = NST * TILE_BYTES;
constexpr int MAXC = 16;              // blocks of a cluster
constexpr int NMETA = 16;             // tiles whose scales are held
constexpr int TERMS = 4;
constexpr int SBUF = 4;                // buffers of scores in tensor memory
// SBUF buffers of S and two of O; a power of two
__host__ __device__ constexpr uint32_t tmem_columns(int GH) { return 8 * TERMS * GH; }

struct Params {
  Pool pool;
  const __nv_bfloat16* q;  // [batch][Hq][128]
  __nv_bfloat16* o;
  const int32_t* seq_lens;
  int G, GP, Hkv, max_len, max_tiles, C, C_log2;  // GP: G rounded up to even; C a power of two
  float scale_log2, log2_tau;
  int per_head;
  int32_t* kept_tiles;
  uint32_t* keep_bits;
  int nw;  // words of a keep_bits row
};

// ------------------------------------------------------------------ instructions
// Instruction descriptor of tcgen05.mma kind::f8f6f4, e4m3 operands, float32 sums.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                         uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Descriptor of an operand without swizzle whose rows of sixteen bytes run along M or N: `lbo`
// bytes to the next eight of K, `sbo` to the next sixteen of N.
__device__ __forceinline__ uint64_t sdesc_plain(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)((lbo >> 4) & 0x3FFFu) << 16 |
         (uint64_t)((sbo >> 4) & 0x3FFFu) << 32 | (uint64_t)1u << 46;
}
// N consecutive columns of this thread's TMEM lane: tmem_ld starts the load, and tmem_ready
// (after tmem_wait, which waits for all that were started) hands its registers over.
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[N]) {
  static_assert(N == 16 || N == 32, "");
  if constexpr (N == 32) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
  }
}
__device__ __forceinline__ void tmem_wait() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void tmem_ready(uint32_t (&r)[N]) {
#pragma unroll
  for (int e = 0; e < N; e += 16)
    asm volatile(""
                 : "+r"(r[e]), "+r"(r[e + 1]), "+r"(r[e + 2]), "+r"(r[e + 3]), "+r"(r[e + 4]),
                   "+r"(r[e + 5]), "+r"(r[e + 6]), "+r"(r[e + 7]), "+r"(r[e + 8]), "+r"(r[e + 9]),
                   "+r"(r[e + 10]), "+r"(r[e + 11]), "+r"(r[e + 12]), "+r"(r[e + 13]),
                   "+r"(r[e + 14]), "+r"(r[e + 15]));
}
// The largest of a warp's values, in every lane; a NaN is passed over.
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
// Whether any softmax thread's predicate holds (a barrier of theirs).
__device__ __forceinline__ bool any_of_softmax(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void sync_softmax() {
  asm volatile("barrier.cta.sync 1, 128;" ::: "memory");
}
__device__ __forceinline__ uint32_t f16x2_to_e4m3x2(__half2 h) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<uint32_t*>(&h)));
  return r;
}
__device__ __forceinline__ __half2 e4m3x2_to_half2(uint32_t x) {
  const uint32_t h = paged::e4m3x2_to_f16x2(x);
  return *reinterpret_cast<const __half2*>(&h);
}
__device__ __forceinline__ float lg2_approx(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The cluster's barrier, for threads that need not be together with their warp's others.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// ------------------------------------------------------------------ shared memory
// What the softmax threads need to know of a tile: its first position, the heads
// that keep it, and the scales of each sixteen tokens (0 where there are none).
struct alignas(16) Meta {
  int pos;
  uint32_t heads;
  int pad[2];
  float k[8], v[8];
};

// What the cluster's blocks send each other at the end.
struct Join {
  float recv[GMAX * (D + MAXC)];  // partial outputs of this block's dimensions, by sender
  float2 ml[MAXC][GMAX];
  int bad[MAXC];
};

template <int GH>
struct Shared {
  unsigned char p[2][T * TERMS * GH];  // P of a tile: key k's terms in rows of sixteen bytes
  unsigned char q[TERMS * GH * D];     // q's terms [term][head][128], 128-byte swizzle
  Meta meta[NMETA];
  float2 part[2][SBUF][4][GH];         // tiles' statistics by warp
  uint64_t full[NST], empty[NST];
  uint64_t s_full[SBUF], s_empty[SBUF], p_full[2], o_full[2], o_empty[2];
  float undo[GMAX];                    // what a head's products are multiplied with
  float mfin[GMAX], lfin[GMAX];        // final max (log2 units) and mass
  float bound[GMAX];
  float wm[4][GMAX];
  int bad, abort, items;
  uint32_t tmem;
  alignas(16) Join join;
};

// Shared memory behind the ring and Shared: statistics [slots][GP] of tiles t = slot C + rank, the
// keep bits [units][words], this block's items.
__host__ __device__ inline int rule_slots(int max_tiles, int C) { return (max_tiles + C - 1) / C; }
__host__ __device__ inline int rule_words(int max_tiles) { return (max_tiles + 31) / 32; }
inline size_t smem_bytes(int G, int max_tiles, int C, bool per_head, bool rule) {
  const int GP = (G + 1) & ~1;
  size_t n = RING + (G > 4 ? sizeof(Shared<8>) : sizeof(Shared<4>));
  if (rule)
    n += (size_t)rule_slots(max_tiles, C) * (GP * sizeof(float2) + sizeof(uint32_t)) +
         (size_t)rule_words(max_tiles) * (per_head ? G : 1) * sizeof(uint32_t);
  return n;
}
constexpr size_t MAX_SMEM = 224 * 1024;

// ------------------------------------------------------------------ pieces of the kernel
// q's terms into shared memory: sixteen threads a head, eight dimensions each. `raw` was
// loaded by thread tid for head tid / 16 (zero for a head that is not there).
template <int GH>
__device__ __forceinline__ void split_q(const uint4& raw, Shared<GH>& sh, float scale_log2) {
  const int tid = threadIdx.x, g = tid >> 4, c = tid & 15;
  float x[8];
  paged::unpack8(raw, x);
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
  if (g >= GH) return;
  int e = (int)(__float_as_uint(amax) >> 23);  // biased exponent
  e = e < 8 ? 8 : (e > 254 ? 254 : e);
  const float up = __uint_as_float((uint32_t)(261 - e) << 23);
  if (c == 0) sh.undo[g] = __uint_as_float((uint32_t)(e - 7) << 23) * scale_log2;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] *= up;
    if (!(fabsf(x[i]) < 512.f)) x[i] = __int_as_float(0x7fc00000);  // infinity: e4m3 has none
  }
#pragma unroll
  for (int k = 0; k < TERMS; ++k) {
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float* y = x + 4 * h;
      w[h] = paged::floats_to_e4m3x2(y[0], y[1]) | paged::floats_to_e4m3x2(y[2], y[3]) << 16;
      const float2 lo = paged::f16x2_to_float2(paged::e4m3x2_to_f16x2(w[h]));
      const float2 hi = paged::f16x2_to_float2(paged::e4m3x2_hi_to_f16x2(w[h]));
      y[0] = (y[0] - lo.x) * 16.f;
      y[1] = (y[1] - lo.y) * 16.f;
      y[2] = (y[2] - hi.x) * 16.f;
      y[3] = (y[3] - hi.y) * 16.f;
    }
    const int n = k * GH + g;
    *reinterpret_cast<uint2*>(sh.q + n * 128 + (((c >> 1) ^ (n & 7)) << 4) + (c & 1) * 8) =
        make_uint2(w[0], w[1]);
  }
}

// The four terms' columns of a row joined, per head.
template <int GH>
__device__ __forceinline__ void join_terms(const uint32_t (&v)[TERMS * GH], float (&x)[GH]) {
#pragma unroll
  for (int g = 0; g < GH; ++g) {
    x[g] = __uint_as_float(v[3 * GH + g]);
#pragma unroll
    for (int k = 2; k >= 0; --k) x[g] = fmaf(x[g], 1.f / 16.f, __uint_as_float(v[k * GH + g]));
  }
}

// A key's probabilities (scaled by 2^8) as e4m3 terms into its row of P. The first term is taken
// from float32; what it leaves of a value in [2^e, 2^(e+1)) is at most 2^(e-4), and goes on in f16,
// rounded by at most 2^(e-16).
template <int GH>
__device__ __forceinline__ void store_p(unsigned char* buf, int key, const float (&p)[GH]) {
  uint32_t w[TERMS][GH / 4];
  const __half2 up = __float2half2_rn(16.f), down = __float2half2_rn(-16.f);
#pragma unroll
  for (int j = 0; j < GH / 2; ++j) {
    uint32_t t = paged::floats_to_e4m3x2(p[2 * j], p[2 * j + 1]);
    const float2 f = __half22float2(e4m3x2_to_half2(t));
    __half2 h = __hmul2(__floats2half2_rn(p[2 * j] - f.x, p[2 * j + 1] - f.y), up);
#pragma unroll
    for (int k = 0; k < TERMS; ++k) {
      if (k > 0) t = f16x2_to_e4m3x2(h);
      w[k][j / 2] = (j & 1) ? w[k][j / 2] | t << 16 : t;
      if (k > 0 && k + 1 < TERMS) h = __hfma2(e4m3x2_to_half2(t), down, __hmul2(h, up));
    }
  }
  const uint32_t* x = &w[0][0];
#pragma unroll
  for (int n = 0; n < TERMS * GH / 16; ++n)
    *reinterpret_cast<uint4*>(buf + n * (T * 16) + key * 16) =
        make_uint4(x[4 * n], x[4 * n + 1], x[4 * n + 2], x[4 * n + 3]);
}

// The table's entry for the lane's first page, before anything is known of the sequence.
constexpr int kNone = -2;
__device__ __forceinline__ int early_page(const Pool& pool, int b, int C, uint32_t rank) {
  const int who = (threadIdx.x >> 5) == W_LOAD ? 0 : 1, lane = threadIdx.x & 31;
  const int per_log2 = 7 - pool.page_log2;
  const long long tile = (long long)(who + 2 * (lane >> per_log2)) * C + rank;
  const long long slot = (tile << per_log2) + (lane & ((1 << per_log2) - 1));
  return slot < pool.max_pages ? pool.table[(long long)b * pool.table_stride + slot] : -1;
}

// A load warp: every second tile (`who`: the even or the odd ones) into the ring, one after
// the other. `place(i)`: the i-th tile's first position and heads. VALUES: a tile's V follows
// its K. `seq0`: stages used before. `early`: the table's entry for the lane's first page of the
// block's own tiles, read side by side with the sequence's length (kNone: not read).
template <bool VALUES, typename Sh, typename Place>
__device__ __forceinline__ bool load_tiles(const Pool& pool, const CUtensorMap* tmK,
                                           const CUtensorMap* tmV, unsigned char* ring, Sh& sh,
                                           int b, int h, int len, int tiles, uint32_t seq0,
                                           uint32_t meta0, int early, Place place) {
  const int who = (threadIdx.x >> 5) == W_LOAD ? 0 : 1;
  const int lane = threadIdx.x & 31;
  const int per_log2 = 7 - pool.page_log2, per = 1 << per_log2;  // pages of a tile
  const int batch = 32 >> per_log2, sub = lane & (per - 1);
  const int32_t* row = pool.table + (long long)b * pool.table_stride;
  volatile int* abort = &sh.abort;
  for (int i0 = who; i0 < tiles; i0 += 2 * batch) {
    // 32 pages at a time, a lane each
    const int i = i0 + 2 * (lane >> per_log2);
    int pos = 0, id = -1;
    uint32_t heads = 0;
    float ks = 0.f, vs = 0.f;
    if (i < tiles) {
      place(i, pos, heads);
      const int at = pos + sub * pool.page, slot = at >> pool.page_log2;
      if (at < len) {
        if (early != kNone && i0 == who)
          id = early;
        else if (slot < pool.max_pages)
          id = row[slot];
        if ((unsigned)id >= (unsigned)pool.num_pages) {
          record_bad_page(0x500);
          sh.bad = 1;
          id = -1;
        }
      }
      if (id >= 0) {
        ks = pool.k_scale[(long long)id * pool.Hkv + h];
        if (VALUES) vs = pool.v_scale[(long long)id * pool.Hkv + h];
      }
    }
    const int n = min(batch, (tiles - i0 + 1) >> 1);
    for (int j = 0; j < n; ++j) {
      uint32_t seq = seq0 + (uint32_t)((VALUES ? 2 : 1) * (i0 + 2 * j));
      const bool mine = (lane >> per_log2) == j;
      const uint32_t bytes =
          (uint32_t)__popc(__ballot_sync(0xffffffffu, mine && id >= 0)) * (uint32_t)pool.page * D;
      for (int w = 0; w < (VALUES ? 2 : 1); ++w, ++seq) {
        const uint32_t st = seq % NST, turn = seq / NST;
        bool ok = true;
        if (lane == 0 && turn > 0)
          ok = mbar_wait(smem_u32(&sh.empty[st]), (turn - 1) & 1, abort, 0x511);
        if (!__shfl_sync(0xffffffffu, (int)ok, 0)) return false;
        if (mine && id >= 0)
          sm100::tma_load_4d(smem_u32(ring) + st * TILE_BYTES + (uint32_t)(sub * pool.page) * D,
                             w ? tmV : tmK, 0, 0, h, id, smem_u32(&sh.full[st]));
        // the scales may still be on their way; the tile counts as there behind them (the bytes may
        // come before they are expected: the phase waits for the arrival)
        if (mine && w == 0) {  // sixteen tiles are held, the softmax is ten behind at most
          Meta& m = sh.meta[(meta0 + (uint32_t)(i0 + 2 * j)) % NMETA];
          if (sub == 0) {
            m.pos = pos;
            m.heads = heads;
          }
          for (int u = 0; u < (8 >> per_log2); ++u) {
            m.k[(sub << (3 - per_log2)) + u] = ks;
            m.v[(sub << (3 - per_log2)) + u] = vs;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_expect_tx(smem_u32(&sh.full[st]), bytes);
      }
    }
  }
  return true;
}

// The warp that issues the products runs as one, so that descriptors and addresses stay in uniform
// registers, and elects a lane for each group of instructions (a single thread's loop took 420
// cycles to issue a tile's, which bounded a block's rate).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(p));
  return p != 0;
}
// Waits for two barriers; what is mostly there already costs one look at both.
__device__ __forceinline__ bool wait_both(uint32_t bar0, uint32_t parity0, uint32_t bar1,
                                          uint32_t parity1, volatile int* abort, unsigned where) {
  const bool ok0 = sm100::mbar_try_wait(bar0, parity0), ok1 = sm100::mbar_try_wait(bar1, parity1);
  return (ok0 || mbar_wait(bar0, parity0, abort, where)) &&
         (ok1 || mbar_wait(bar1, parity1, abort, where));
}
struct Issuer {
  uint64_t k, v, q, p;  // descriptors of ring stage 0 as keys and as values, of q and of P
  uint32_t tmem;
};
// S of the tile in ring stage `seq` into S buffer s % SBUF:
template <int GH>
__device__ __forceinline__ bool issue_s(Shared<GH>& sh, const Issuer& is, uint32_t seq, uint32_t s) {
  constexpr uint32_t ID = idesc_e4m3(T, TERMS * GH, false, false);
  volatile int* abort = &sh.abort;
  const uint32_t st = seq % NST, buf = s % SBUF;
  // a barrier that nothing has used yet counts as through with the phase before its first
  const bool ok = wait_both(smem_u32(&sh.full[st]), (seq / NST) & 1, smem_u32(&sh.s_empty[buf]),
                            (s / SBUF + 1) & 1, abort, 0x512);
  if (!__all_sync(0xffffffffu, ok)) return false;
  sm100::tc_fence_after();
  if (elect_one()) {
    const uint64_t a = is.k + st * (TILE_BYTES >> 4);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
      mma_e4m3(is.tmem + buf * (TERMS * GH), a + 2 * kk, is.q + 2 * kk, ID, kk > 0);
    sm100::mma_commit(smem_u32(&sh.empty[st]));  // first: behind the other the block may end
    sm100::mma_commit(smem_u32(&sh.s_full[buf]));
  }
  __syncwarp();
  return true;
}
// O of the i-th tile with values, V in ring stage `seq`:
template <int GH>
__device__ __forceinline__ bool issue_o(Shared<GH>& sh, const Issuer& is, uint32_t seq, uint32_t i) {
  constexpr uint32_t ID = idesc_e4m3(T, TERMS * GH, true, true);
  volatile int* abort = &sh.abort;
  const uint32_t st = seq % NST, buf = i & 1;
  bool ok = wait_both(smem_u32(&sh.full[st]), (seq / NST) & 1, smem_u32(&sh.o_empty[buf]),
                      ((i >> 1) + 1) & 1, abort, 0x515);
  ok = ok && mbar_wait(smem_u32(&sh.p_full[buf]), (i >> 1) & 1, abort, 0x514);
  if (!__all_sync(0xffffffffu, ok)) return false;
  sm100::tc_fence_after();
  if (elect_one()) {
    const uint64_t a = is.v + st * (TILE_BYTES >> 4), b = is.p + buf * (T * TERMS * GH >> 4);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)  // 32 keys a step: 4 KB of V, 512 bytes of P
      mma_e4m3(is.tmem + (SBUF + buf) * (TERMS * GH), a + 256 * kk, b + 32 * kk, ID, kk > 0);
    sm100::mma_commit(smem_u32(&sh.empty[st]));  // first: behind the other the block may end
    sm100::mma_commit(smem_u32(&sh.o_full[buf]));
  }
  __syncwarp();
  return true;
}
// Scores two tiles ahead of the values. `held`: the scores are there from before, and the i-th
// tile is the block's held[i].
template <int GH>
__device__ __forceinline__ bool issue_pairs(Shared<GH>& sh, const Issuer& is, int tiles, uint32_t seq0,
                                            uint32_t s0, const uint32_t* held) {
  bool ok = true;
  if (held) {
    for (int i = 0; i < tiles && ok; ++i)
      ok = issue_o<GH>(sh, is, seq0 + 2 * (held[i] & 0xffffffu) + 1, i);
    return ok;
  }
  for (int i = 0; i < 2 && i < tiles && ok; ++i) ok = issue_s<GH>(sh, is, seq0 + 2 * i, s0 + i);
  for (int i = 0; i < tiles && ok; ++i) {
    ok = issue_o<GH>(sh, is, seq0 + 2 * i + 1, i);
    if (ok && i + 2 < tiles) ok = issue_s<GH>(sh, is, seq0 + 2 * (i + 2), s0 + i + 2);
  }
  return ok;
}

// A softmax warp's wait. When it runs out the warp goes on all the same, over whatever lies
// there: the others wait for it at their barriers, and the call is reported as timed out.
__device__ __forceinline__ void warp_wait(uint64_t* bar, uint32_t parity, int* abort,
                                          unsigned where) {
  mbar_wait(smem_u32(bar), parity, abort, where);
  __syncwarp();
}

// A softmax warp is through with a buffer.
__device__ __forceinline__ void release(uint64_t* bar) {
  sm100::tc_fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(bar));
}

// Scores of this thread's key in log2 units, -inf behind the sequence, of the tile whose
// products `v` holds.
template <int GH>
__device__ __forceinline__ void scores(const uint32_t (&v)[TERMS * GH], float ks, int left,
                                       const float (&undo)[GH], float (&x)[GH]) {
  join_terms<GH>(v, x);
#pragma unroll
  for (int g = 0; g < GH; ++g) x[g] = (int)threadIdx.x < left ? x[g] * (undo[g] * ks) : kNegInf;
}
// The S-th tile's products, when they are there.
template <int GH>
__device__ __forceinline__ void start_scores(Shared<GH>& sh, uint32_t s, uint32_t (&v)[TERMS * GH]) {
  warp_wait(&sh.s_full[s % SBUF], (s / SBUF) & 1, &sh.abort, 0x517);
  sm100::tc_fence_after();
  tmem_ld(sh.tmem + (s % SBUF) * (TERMS * GH) + ((threadIdx.x >> 5) << 21), v);
}

// out += O of the i-th tile, f[g] times, for the heads that keep it (a value that is NaN
// shows only in those).
template <int GH>
__device__ __forceinline__ void add_o(Shared<GH>& sh, uint32_t i, const float (&f)[GH],
                                      uint32_t heads, float (&out)[GH]) {
  const uint32_t buf = i & 1;
  warp_wait(&sh.o_full[buf], (i >> 1) & 1, &sh.abort, 0x518);
  sm100::tc_fence_after();
  uint32_t v[TERMS * GH];
  tmem_ld(sh.tmem + (SBUF + buf) * (TERMS * GH) + ((threadIdx.x >> 5) << 21), v);
  tmem_wait();
  tmem_ready(v);
  release(&sh.o_empty[buf]);
  float x[GH];
  join_terms<GH>(v, x);
#pragma unroll
  for (int g = 0; g < GH; ++g)
    if ((heads >> g) & 1u) out[g] = fmaf(x[g], f[g], out[g]);
}

// The softmax threads' part of the tiles with values. FIXED: `mref` is the rows' final
// max; else it runs along, and l is the mass of this thread's keys.
template <int GH, bool FIXED>
__device__ __forceinline__ void softmax_pv(Shared<GH>& sh, unsigned char* ring, int len, int tiles,
                                           uint32_t s0, uint32_t seq0, const uint32_t* held,
                                           const float (&undo)[GH], float (&mref)[GH],
                                           float (&l)[GH], float (&out)[GH]) {
  const int key = threadIdx.x, warp = key >> 5;
  float f[GH];  // the tile before: what its O counts
#pragma unroll
  for (int g = 0; g < GH; ++g) f[g] = 0.f;
  uint32_t heads_before = 0;
  for (int i = 0; i < tiles; ++i) {
    const uint32_t nth = FIXED && held ? held[i] & 0xffffffu : (uint32_t)i;
    const uint32_t s = s0 + nth;
    const Meta& m = sh.meta[s % NMETA];
    uint32_t raw[TERMS * GH];
    start_scores<GH>(sh, s, raw);
    // what is wanted of m is read before the products' buffer is given back: the load warp may
    // overwrite it later
    const float ks = m.k[key >> 4];
    const int left = len - m.pos;
    const uint32_t heads = FIXED ? (held ? held[i] >> 24 : m.heads) : 0xffu;
    // pages of different scales: V's bytes count u, the largest, and P takes the rest
    const float4 v0 = *reinterpret_cast<const float4*>(m.v);
    const float4 v1 = *reinterpret_cast<const float4*>(m.v + 4);
    const float vs = m.v[key >> 4];
    const float u = fmaxf(fmaxf(fmaxf(fabsf(v0.x), fabsf(v0.y)), fmaxf(fabsf(v0.z), fabsf(v0.w))),
                          fmaxf(fmaxf(fabsf(v1.x), fabsf(v1.y)), fmaxf(fabsf(v1.z), fabsf(v1.w))));
    const float ratio = vs == u ? 1.f : (vs == 0.f ? 0.f : vs / u);
    float x[GH];
    tmem_wait();
    tmem_ready(raw);
    release(&sh.s_empty[s % SBUF]);
    scores<GH>(raw, ks, left, undo, x);
    if (!FIXED) {
      bool above = false;
#pragma unroll
      for (int g = 0; g < GH; ++g) above |= x[g] > mref[g];
      if (any_of_softmax(above)) {
#pragma unroll
        for (int g = 0; g < GH; ++g) {
          const float top = warp_max(x[g]);
          if ((key & 31) == 0) sh.wm[warp][g] = top;
        }
        sync_softmax();
#pragma unroll
        for (int g = 0; g < GH; ++g) {
          const float top = fmaxf(fmaxf(sh.wm[0][g], sh.wm[1][g]), fmaxf(sh.wm[2][g], sh.wm[3][g]));
          const float now = fmaxf(mref[g], top);
          const float c = mref[g] == kNegInf ? 0.f : ex2_approx(mref[g] - now);
          mref[g] = now;
          l[g] *= c;
          out[g] *= c;
          f[g] *= c;
        }
      }
    }
    float p[GH];
#pragma unroll
    for (int g = 0; g < GH; ++g) {
      if (FIXED && !((heads >> g) & 1u)) x[g] = kNegInf;
      const float z = (mref[g] == kNegInf ? 0.f : mref[g]) - 8.f;
      p[g] = ex2_approx(x[g] - z);
      if (!FIXED) l[g] += p[g];
      p[g] *= ratio;
    }
    store_p<GH>(sh.p[i & 1], key, p);
    if (left < T) {
      // rows behind the sequence hold anything, and a product with a NaN is NaN even where P
      // is zero
      const uint32_t seq = seq0 + 2u * nth + 1u, st = seq % NST;
      warp_wait(&sh.full[st], (seq / NST) & 1, &sh.abort, 0x519);
      if (key >= left)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          reinterpret_cast<uint4*>(ring + st * TILE_BYTES + key * D)[e] = make_uint4(0, 0, 0, 0);
    }
    sm100::fence_proxy_async_smem();
    __syncwarp();
    if ((key & 31) == 0) mbar_arrive(smem_u32(&sh.p_full[i & 1]));
    if (i > 0) add_o<GH>(sh, i - 1, f, heads_before, out);
    heads_before = heads;
#pragma unroll
    for (int g = 0; g < GH; ++g) f[g] = u * (1.f / 256.f);
  }
  if (tiles > 0) add_o<GH>(sh, tiles - 1, f, heads_before, out);
}

template <int GH>
__device__ __forceinline__ void free_tmem(const Shared<GH>& sh) {
  __syncwarp();
  sm100::tc_fence_after();
  sm100::tmem_dealloc(sh.tmem, tmem_columns(GH));
}

// Joins the blocks' outputs and writes o = sum / l: thread tid of the softmax warps has
// dimension tid of every head. dense: the blocks' references differ (sh.mfin), else
// sh.lfin is the whole cluster's mass. Each block owns some of the dimensions, and the others
// write their partial sums of them into its shared memory: no round trips.
template <int GH>
__device__ __forceinline__ void join_and_store(const Params& p, Shared<GH>& sh,
                                               const float (&out)[GH], uint32_t rank,
                                               __nv_bfloat16* o, bool dense) {
  const int tid = threadIdx.x, C = p.C, G = p.G;
  Join& jn = sh.join;
  const float nan = __int_as_float(0x7fc00000);
  if (C == 1) {
    if ((tid >> 5) == W_TMEM) free_tmem(sh);
    if (tid < NC)
#pragma unroll
      for (int g = 0; g < GH; ++g)
        if (g < G) o[g * D + tid] = __float2bfloat16_rn(sh.bad ? nan : out[g] / sh.lfin[g]);
    return;
  }
  const int each = (D + C - 1) / C;  // dimensions a block owns
  if (tid < NC) {
    const int owner = tid / each, i = tid - owner * each;
#pragma unroll
    for (int g = 0; g < GH; ++g)
      if (g < G)
        sm100::st_cluster_f32(
            sm100::mapa_rank(smem_u32(&jn.recv[((int)rank * G + g) * each + i]), owner), out[g]);
  } else if (tid < NC + C) {
    sm100::st_cluster_u32(sm100::mapa_rank(smem_u32(&jn.bad[rank]), tid - NC), sh.bad);
  }
  if (dense && tid < GMAX * C) {
    const int g = tid % GMAX;
    sm100::st_cluster_f32x2(sm100::mapa_rank(smem_u32(&jn.ml[rank][g]), tid / GMAX),
                            make_float2(sh.mfin[g], sh.lfin[g]));
  }
  cluster_arrive();
  // given back here, by a warp whose lanes are together (behind the loop below they need not be,
  // and a deallocation by part of a warp never ends)
  if ((tid >> 5) == W_TMEM) free_tmem(sh);
  cluster_wait();
  for (int e = tid; e < G * each; e += NT) {
    const int g = e / each, i = e - g * each, dim = (int)rank * each + i;
    if (dim >= D) continue;
    float sum = 0.f, l = dense ? 0.f : sh.lfin[g], top = kNegInf;
    int bad = 0;
    if (dense)
      for (int k = 0; k < C; ++k) top = fmaxf(top, jn.ml[k][g].x);
    for (int k = 0; k < C; ++k) {
      float f = 1.f;
      if (dense) {
        const float2 ml = jn.ml[k][g];
        f = ml.x == kNegInf ? 0.f : ex2_approx(ml.x - top);
        l += f * ml.y;
      }
      sum += f * jn.recv[k * G * each + e];
      bad |= jn.bad[k];
    }
    o[g * D + dim] = __float2bfloat16_rn(bad ? nan : sum / l);
  }
}

// An unused slot of the batch, or a length that the call did not allow for:
// the output without any work. True when there is nothing else to do.
__device__ __forceinline__ bool trivial(const Params& p, long long grp, int len, uint32_t rank,
                                        __nv_bfloat16* o) {
  const bool fits = len <= p.max_len;
  if (len > 0 && fits) return false;
  if (rank == 0) {
    const int tid = threadIdx.x, units = p.per_head ? p.G : 1;
    if (!fits && tid == 0) record_bad_page(0x510);
    const __nv_bfloat16 z = __float2bfloat16_rn(fits ? 0.f : __int_as_float(0x7fc00000));
    for (int e = tid; e < p.G * D; e += NT) o[e] = z;
    if (p.kept_tiles && tid < units) p.kept_tiles[grp * units + tid] = 0;
    if (p.keep_bits)
      for (int e = tid; e < units * p.nw; e += NT) p.keep_bits[grp * units * p.nw + e] = 0u;
  }
  return true;
}

// A head's running max and mass over the kept tiles, and the least tile max that is kept.
struct Walk {
  float m, l, bound;
  __device__ __forceinline__ void take(float2 s, float thr) {
    const float d = s.x - m;
    const bool up = !(d <= 0.f);  // a NaN, too
    const float f = ex2_approx(m == kNegInf ? kNegInf : -fabsf(d));  // the smaller one's share
    l = up ? fmaf(l, f, s.y) : fmaf(s.y, f, l);
    m = up ? s.x : m;
    bound = m + lg2_approx(l) + thr;
  }
};

// Phase B: replays the rule over the cluster's statistics, newest first, in stretches that
// fit in the ring's space (a single block's statistics lie in tile order already); leaves the
// rows' final max and mass, the keep bits, and this block's list of tiles.
//
// A head's bound never falls, so a tile below the bound as it stands now is out for good: the
// warps sort out, side by side, those that no head could still want at the bound that the newest
// 32 tiles left, and only the others are looked at one by one (vote and update, about 300
// cycles each). A NaN score is below no bound and leaves one that nothing is below: its tile is
// kept, and every older one, sorted out or not. Group: one warp, a lane per head. Per head: a
// warp per head.
template <int GH>
__device__ __forceinline__ void replay_rule(const Params& p, Shared<GH>& sh, unsigned char* smem,
                                            bool resident, float2* stats, uint32_t* keep,
                                            uint32_t* list, long long grp, int len, int nt,
                                            uint32_t rank) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = p.G, GP = p.GP, C = p.C;
  const int units = p.per_head ? G : 1, words = rule_words(p.max_tiles);
  const float2* loc = C > 1 ? reinterpret_cast<const float2*>(smem) : stats;
  const int cap = C > 1 ? ((int)(RING / sizeof(float2)) / GP) & ~31 : 0x7fffffe0;
  const uint32_t stats_a = smem_u32(stats);
  const float thr = p.log2_tau - lg2_approx((float)len);
  const int unit = p.per_head ? warp : 0;  // whose tiles this warp walks
  const bool walks = p.per_head ? warp < G : warp == 0;
  const int head = p.per_head ? warp : lane & 7;
  const int seen = head < G ? head : G - 1;  // lanes without a head follow one that is there
  Walk w = {kNegInf, 0.f, kNegInf};
  for (int hi = nt; hi > 0;) {
    const int lo = hi > cap ? (hi - cap + 31) & ~31 : 0;
    if (C > 1) {
      const int per = GP / 2, n = (hi - lo) * per;  // pieces of sixteen bytes
      for (int e0 = tid; e0 < n; e0 += 4 * NT) {
        float4 x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int e = e0 + u * NT;
          if (e >= n) break;
          const int t = lo + e / per, slot = t >> p.C_log2;
          x[u] = sm100::ld_cluster_f32x4(sm100::mapa_rank(
              stats_a + 16u * (uint32_t)(slot * per + e % per), (uint32_t)(t & (C - 1))));
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int e = e0 + u * NT;
          if (e < n) reinterpret_cast<float4*>(smem)[e] = x[u];
        }
      }
      __syncwarp();
      __syncthreads();
    }
    const int last = (hi - 1) >> 5, first = lo >> 5;
    // the tiles of word wi that are `open`, newest first; the word comes out as what is kept.
    // `all`: take the newest of them whatever it is, and sort the rest out at its bound.
    auto walk = [&](int wi, uint32_t open, bool all) {
      const float2* at = loc + (size_t)(wi * 32 - lo) * GP;
      uint32_t word = 0;
      if (all) {
        const int bit = 31 - __clz(open);
        word = 1u << bit;
        w.take(at[bit * GP + seen], thr);
        if (!p.per_head) {
          if (lane < G) sh.bound[lane] = w.bound;
          __syncwarp();
        }
        bool may = false;
        if (lane < bit) {
          if (p.per_head) {
            may = !(at[lane * GP + head].x < w.bound);
          } else {
#pragma unroll
            for (int g = 0; g < GH; ++g)
              if (g < G) may |= !(at[lane * GP + g].x < sh.bound[g]);
          }
        }
        open = __ballot_sync(0xffffffffu, may);
      }
      int bit = 31 - __clz(open | 1u);
      float2 x = at[bit * GP + seen];
      while (open) {
        // behind a NaN nothing is below the bound, whatever has been sorted out
        const bool lost = __any_sync(0xffffffffu, isnan(x.x));
        open = lost ? (1u << bit) - 1u : open & ~(1u << bit);
        const int next = 31 - __clz(open | 1u);
        const float2 y = at[next * GP + seen];  // on its way while this one is decided
        // nearly every tile that is left is kept: what it would make of the state is worked out
        // beside the vote, and taken over without a branch
        Walk kept = w;
        kept.take(x, thr);
        const bool take = __any_sync(0xffffffffu, !(x.x < w.bound));  // a NaN keeps
        word |= (take ? 1u : 0u) << bit;
        w.m = take ? kept.m : w.m;
        w.l = take ? kept.l : w.l;
        w.bound = take ? kept.bound : w.bound;
        bit = next;
        x = y;
      }
      if (lane == 0) keep[unit * words + wi] = word;
    };
    if (walks) {
      const int in = hi - last * 32;
      walk(last, in >= 32 ? 0xffffffffu : (1u << in) - 1u, hi == nt);
      if (p.per_head ? lane == 0 : lane < G) sh.bound[p.per_head ? warp : lane] = w.bound;
    }
    __syncwarp();
    if (last > first) __syncthreads();
    for (int wi = first + warp; wi < last; wi += NT / 32) {
      const float2* at = loc + (size_t)(wi * 32 + lane - lo) * GP;
      bool may = false;
#pragma unroll
      for (int g = 0; g < GH; ++g) {
        if (g >= G) break;
        const bool wants = !(at[g].x < sh.bound[g]);
        may |= wants;
        if (p.per_head) {
          const uint32_t open = __ballot_sync(0xffffffffu, wants);
          if (lane == 0) keep[g * words + wi] = open;
        }
      }
      const uint32_t open = __ballot_sync(0xffffffffu, may);
      if (!p.per_head && lane == 0) keep[wi] = open;
    }
    __syncwarp();
    if (last > first) __syncthreads();
    if (walks)
      for (int w0 = last - 1; w0 >= first; w0 -= 32) {  // 32 words at a time, a lane each
        uint32_t done = 0;  // words that need no further look
        const bool there = w0 - lane >= first;
        uint32_t mine = there ? keep[unit * words + w0 - lane] : 0u;
        uint32_t some = __ballot_sync(0xffffffffu, mine != 0u);
        while (true) {
          if (__any_sync(0xffffffffu, isnan(w.bound))) {
            mine = there ? 0xffffffffu : 0u;
            some = __ballot_sync(0xffffffffu, mine != 0u) & ~done;
          }
          if (!some) break;
          const int src = __ffs(some) - 1;
          some &= some - 1;
          done = (2u << src) - 1u;
          walk(w0 - src, __shfl_sync(0xffffffffu, mine, src), false);
        }
      }
    hi = lo;
    __syncwarp();
    if (hi > 0) __syncthreads();
  }
  if (p.per_head ? (warp < G && lane == 0) : tid < G) {
    const int g = p.per_head ? warp : tid;
    sh.mfin[g] = w.m == kNegInf ? 0.f : w.m;
    sh.lfin[g] = w.l;
  }
  __syncwarp();
  __syncthreads();
  const int live = (nt + 31) / 32;
  if (warp == 0 && resident) {  // its own tiles, as many as are kept
    const int t = lane * C + (int)rank;
    uint32_t heads = 0;
    if (lane < 2 && t < nt)
      for (int u = 0; u < units; ++u)
        if ((keep[u * words + (t >> 5)] >> (t & 31)) & 1u) heads |= p.per_head ? 1u << u : 0xffu;
    const uint32_t kept = __ballot_sync(0xffffffffu, heads != 0u);
    if (heads) list[__popc(kept & ((1u << lane) - 1u))] = (uint32_t)lane | heads << 24;
    if (lane == 0) sh.items = __popc(kept);
  } else if (warp == 0) {  // the n-th kept tile (in the order of positions) is block n mod C's
    int count = 0;
    for (int w0 = 0; w0 < live; w0 += 32) {
      uint32_t any = 0;
      if (w0 + lane < live)
        for (int u = 0; u < units; ++u) any |= keep[u * words + w0 + lane];
      uint32_t some = __ballot_sync(0xffffffffu, any != 0u);
      while (some) {  // a word with kept tiles, a lane each
        const int src = __ffs(some) - 1, wi = w0 + src;
        some &= some - 1;
        const uint32_t word = __shfl_sync(0xffffffffu, any, src);
        const int n = count + __popc(word & ((1u << lane) - 1u));
        if (((word >> lane) & 1u) && (n & (C - 1)) == (int)rank) {
          uint32_t heads = 0xffu;
          if (p.per_head) {
            heads = 0;
            for (int u = 0; u < units; ++u) heads |= ((keep[u * words + wi] >> lane) & 1u) << u;
          }
          list[n >> p.C_log2] = (uint32_t)(wi * 32 + lane) | heads << 24;
        }
        count += __popc(word);
      }
    }
    if (lane == 0) sh.items = (count - (int)rank + C - 1) >> p.C_log2;
  } else if (rank == 0) {
    if (p.kept_tiles)
      for (int u = warp - 1; u < units; u += NT / 32 - 1) {
        int n = 0;
        for (int e = lane; e < live; e += 32) n += __popc(keep[u * words + e]);
        n = __reduce_add_sync(0xffffffffu, n);
        if (lane == 0) p.kept_tiles[grp * units + u] = n;
      }
    if (p.keep_bits)
      for (int e = tid - 32; e < units * p.nw; e += NT - 32) {
        const int u = e / p.nw, wi = e - u * p.nw;
        p.keep_bits[grp * units * p.nw + e] = wi < live ? keep[u * words + wi] : 0u;
      }
  }
  sm100::fence_proxy_async_smem();  // the ring's space goes back to the TMA
  __syncwarp();
  __syncthreads();
}

// ------------------------------------------------------------------ the kernel
template <int GH, bool RULE>
__global__ void __launch_bounds__(NT, 2) decode_kernel(const __grid_constant__ CUtensorMap tmK,
                                                       const __grid_constant__ CUtensorMap tmV,
                                                       const Params p) {
  constexpr uint32_t TCOLS = tmem_columns(GH);
  static_assert(SBUF + 2 <= 8 && 2 * TCOLS <= 512, "two blocks share an SM's tensor memory");
  extern __shared__ unsigned char smem[];
  Shared<GH>& sh = *reinterpret_cast<Shared<GH>*>(smem + RING);
  if (smem_u32(smem) & 1023u) {  // the swizzle needs it; without static shared memory it holds
    if (threadIdx.x == 0) record_layout_error(0x51f);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = p.G, C = p.C;
  const Pool& pool = p.pool;
  const uint32_t rank = blockIdx.x;
  const int h = blockIdx.y, b = blockIdx.z;
  const long long grp = (long long)b * p.Hkv + h;
  __nv_bfloat16* o = p.o + grp * G * D;

  const int len = p.seq_lens[b];
  int early = kNone;
  if (warp == W_LOAD || warp == W_LOAD2) early = early_page(pool, b, C, rank);
  uint4 qraw = make_uint4(0, 0, 0, 0);
  if (tid < NC && (tid >> 4) < G)
    qraw = *reinterpret_cast<const uint4*>(p.q + grp * G * D + tid * 8);
  if (warp == W_LOAD) {
    if (lane == 0) {
      for (int s = 0; s < NST; ++s) {
        sm100::mbar_init(smem_u32(&sh.full[s]), 1);
        sm100::mbar_init(smem_u32(&sh.empty[s]), 1);
      }
      for (int s = 0; s < SBUF; ++s) {
        sm100::mbar_init(smem_u32(&sh.s_full[s]), 1);
        sm100::mbar_init(smem_u32(&sh.s_empty[s]), 4);
      }
      for (int s = 0; s < 2; ++s) {
        sm100::mbar_init(smem_u32(&sh.o_full[s]), 1);
        sm100::mbar_init(smem_u32(&sh.o_empty[s]), 4);
        sm100::mbar_init(smem_u32(&sh.p_full[s]), 4);
      }
      sm100::fence_mbar_init();
      sh.bad = sh.abort = 0;
    }
    __syncwarp();
  }
  __syncthreads();
  if (trivial(p, grp, len, rank, o)) return;
  if (!RULE && C > 1) cluster_arrive();
  const int nt = (int)(((long long)len + T - 1) / T);
  const int tiles = nt > (int)rank ? (nt - (int)rank + C - 1) / C : 0;  // this block's
  const int units = p.per_head ? G : 1, words = rule_words(p.max_tiles);
  float2* stats = reinterpret_cast<float2*>(smem + RING + sizeof(Shared<GH>));  // [slots][GP]
  uint32_t* keep = reinterpret_cast<uint32_t*>(stats + (size_t)p.GP * rule_slots(p.max_tiles, C));
  uint32_t* list = keep + units * words;
  __syncwarp();  // here and below: a warp-wide instruction or barrier wants its lanes together

  auto own_tile = [&](int i, int& pos, uint32_t& heads) {
    pos = (i * C + (int)rank) * T;
    heads = 0xffu;
  };
  bool ok = true;
  float undo[GH], mref[GH], l[GH], out[GH];
#pragma unroll
  for (int g = 0; g < GH; ++g) {
    undo[g] = 0.f;
    mref[g] = kNegInf;
    l[g] = out[g] = 0.f;
  }
  if (warp != W_LOAD && warp != W_LOAD2) {  // the load warps need none of this
    if (warp == W_TMEM) {
      sm100::tmem_alloc(smem_u32(&sh.tmem), TCOLS);
      sm100::tmem_relinquish();
    } else if (warp < 4) {
      split_q<GH>(qraw, sh, p.scale_log2);
      sm100::fence_proxy_async_smem();
    }
    sm100::tc_fence_before();
    __syncwarp();
    asm volatile("barrier.cta.sync 2, 192;" ::: "memory");
    sm100::tc_fence_after();
#pragma unroll
    for (int g = 0; g < GH; ++g) undo[g] = sh.undo[g];
  }
  Issuer issuer;
  issuer.k = sm100::sdesc_sw128(smem_u32(smem), 16, 1024);
  issuer.v = sm100::sdesc_sw128(smem_u32(smem), TILE_BYTES, 1024);
  issuer.q = sm100::sdesc_sw128(smem_u32(sh.q), 16, 1024);
  issuer.p = sdesc_plain(smem_u32(sh.p), 128, T * 16);
  issuer.tmem = warp == W_MMA ? __shfl_sync(0xffffffffu, sh.tmem, 0) : 0u;

  if constexpr (RULE) {
    // ---- A: statistics. A block with at most two tiles loads their values as well and keeps
    // all of it, scores in tensor memory included: C then has nothing to wait for (some values
    // that nobody wants are read, while a block waits for little else than latency).
    const bool resident = nt <= 2 * C;
    if (warp == W_LOAD || warp == W_LOAD2) {
      if (resident)
        ok = load_tiles<true>(pool, &tmK, &tmV, smem, sh, b, h, len, tiles, 0u, 0u, early, own_tile);
      else
        ok = load_tiles<false>(pool, &tmK, &tmV, smem, sh, b, h, len, tiles, 0u, 0u, early, own_tile);
    } else if (warp == W_MMA) {
      for (int i = 0; i < tiles && ok; ++i) ok = issue_s<GH>(sh, issuer, resident ? 2 * i : i, i);
    } else if (warp < 4) {
      // NB tiles at a time: their loads and reductions overlap
      constexpr int NB = GH == 4 ? 4 : 2;
      for (int i = 0; i < tiles; i += NB) {
        uint32_t raw[NB][TERMS * GH];
        float ks[NB] = {};
        int left[NB] = {};
#pragma unroll
        for (int q = 0; q < NB; ++q) {
          if (i + q >= tiles) break;
          start_scores<GH>(sh, i + q, raw[q]);
          const Meta& m = sh.meta[(i + q) % NMETA];
          ks[q] = m.k[tid >> 4];
          left[q] = len - m.pos;
        }
        tmem_wait();
#pragma unroll
        for (int q = 0; q < NB; ++q) {
          tmem_ready(raw[q]);
          if (i + q < tiles) release(&sh.s_empty[(i + q) % SBUF]);
        }
        float x[NB][GH], m[NB][GH];
#pragma unroll
        for (int q = 0; q < NB; ++q) {
          scores<GH>(raw[q], ks[q], left[q], undo, x[q]);
          // a warp's 32 keys; a quarter without a finite score: mass 0
#pragma unroll
          for (int g = 0; g < GH; ++g) {
            m[q][g] = warp_max(x[q][g]);
            x[q][g] = ex2_approx(x[q][g] - (m[q][g] == kNegInf ? 0.f : m[q][g]));
          }
        }
        // sums: each step halves the heads a lane is at work on, lane / (32 / GH) is left with one
#pragma unroll
        for (int n = GH / 2, d = 16; n >= 1; n >>= 1, d >>= 1) {
          const bool up = lane & d;
#pragma unroll
          for (int g = 0; g < n; ++g)
#pragma unroll
            for (int q = 0; q < NB; ++q) {
              const float give = up ? x[q][g] : x[q][g + n];
              x[q][g] = (up ? x[q][g + n] : x[q][g]) + __shfl_xor_sync(0xffffffffu, give, d);
              m[q][g] = up ? m[q][g + n] : m[q][g];
            }
        }
#pragma unroll
        for (int d = 16 / GH; d >= 1; d >>= 1)
#pragma unroll
          for (int q = 0; q < NB; ++q) x[q][0] += __shfl_xor_sync(0xffffffffu, x[q][0], d);
        auto& part = sh.part[(i / NB) & 1];
        if (lane % (32 / GH) == 0)
#pragma unroll
          for (int q = 0; q < NB; ++q)
            part[q][warp][lane / (32 / GH)] = make_float2(m[q][0], x[q][0]);
        sync_softmax();
        if (warp < NB && i + warp < tiles && lane < G) {  // the quarters' statistics as the tile's
          float2 y[4];
#pragma unroll
          for (int w = 0; w < 4; ++w) y[w] = part[warp][w][lane];
          float top = fmaxf(fmaxf(y[0].x, y[1].x), fmaxf(y[2].x, y[3].x));
          const float z = top == kNegInf ? 0.f : top;
          float sum = 0.f;
#pragma unroll
          for (int w = 0; w < 4; ++w) sum += y[w].y * ex2_approx(y[w].x - z);
          if (isnan(sum)) top = sum;  // a tile with a NaN score is kept, and shows
          stats[(i + warp) * p.GP + lane] = make_float2(top, sum);
        }
        __syncwarp();
      }
    }
    if (sh.abort) sm100::drain_in_flight();
    __syncwarp();
    if (C > 1) {
      cluster_arrive();
      cluster_wait();
    } else {
      __syncthreads();
    }

    // ---- B
    replay_rule<GH>(p, sh, smem + (resident ? 4 * TILE_BYTES : 0), resident, stats, keep, list, grp,
                    len, nt, rank);

    // ---- C: values of this block's kept tiles
    const int items = sh.items;
    const uint32_t done = resident ? 0u : (uint32_t)tiles;
    const uint32_t* held = resident ? list : nullptr;
    if (warp == W_LOAD || warp == W_LOAD2) {
      auto kept_tile = [&](int i, int& pos, uint32_t& heads) {
        const uint32_t x = list[i];
        pos = (int)(x & 0xffffffu) * T;
        heads = x >> 24;
      };
      if (ok && !resident)
        load_tiles<true>(pool, &tmK, &tmV, smem, sh, b, h, len, items, done, done, kNone, kept_tile);
    } else if (warp == W_MMA) {
      if (ok) ok = issue_pairs<GH>(sh, issuer, items, done, done, held);
      // a resident block has asked for the values of all its tiles, and nothing above waits for
      // those of a skipped one: they must have landed before the block's shared memory goes
      for (int i = 0; resident && ok && i < tiles; ++i)
        ok = mbar_wait(smem_u32(&sh.full[2 * i + 1]), 0, &sh.abort, 0x51a);
      __syncwarp();
    } else if (warp < 4) {
#pragma unroll
      for (int g = 0; g < GH; ++g) mref[g] = g < G ? sh.mfin[g] : 0.f;
      softmax_pv<GH, true>(sh, smem, len, items, done, done, held, undo, mref, l, out);
    }
  } else {
    if (warp == W_LOAD || warp == W_LOAD2) {
      ok = load_tiles<true>(pool, &tmK, &tmV, smem, sh, b, h, len, tiles, 0u, 0u, early, own_tile);
    } else if (warp == W_MMA) {
      issue_pairs<GH>(sh, issuer, tiles, 0u, 0u, nullptr);
    } else if (warp < 4) {
      softmax_pv<GH, false>(sh, smem, len, tiles, 0u, 0u, nullptr, undo, mref, l, out);
      // the block's mass per head: every thread has its own keys'
#pragma unroll
      for (int g = 0; g < GH; ++g) {
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) l[g] += __shfl_xor_sync(0xffffffffu, l[g], d);
        if (lane == 0) sh.wm[warp][g] = l[g];
      }
      sync_softmax();
      if (tid == 0)
#pragma unroll
        for (int g = 0; g < GH; ++g) {
          sh.mfin[g] = mref[g];
          sh.lfin[g] = (sh.wm[0][g] + sh.wm[1][g] + sh.wm[2][g] + sh.wm[3][g]) * (1.f / 256.f);
        }
    }
  }
  if (sh.abort) sm100::drain_in_flight();
  sm100::tc_fence_before();
  __syncwarp();
  __syncthreads();
  if (!RULE && C > 1) cluster_wait();  // the other blocks run
  join_and_store<GH>(p, sh, out, rank, o, !RULE);
  if (!RULE && rank == 0) {  // every tile is kept
    if (p.kept_tiles && tid < units) p.kept_tiles[grp * units + tid] = nt;
    if (p.keep_bits)
      for (int e = tid; e < units * p.nw; e += NT) {
        const int left = nt - 32 * (e % p.nw);
        p.keep_bits[grp * units * p.nw + e] =
            left >= 32 ? 0xffffffffu : (left > 0 ? (1u << left) - 1u : 0u);
      }
  }
}

using Kernel = void (*)(CUtensorMap, CUtensorMap, Params);
inline Kernel decode_kernel_of(int G, bool rule) {
  if (G > 4) return rule ? decode_kernel<8, true> : decode_kernel<8, false>;
  return rule ? decode_kernel<4, true> : decode_kernel<4, false>;
}

}  // namespace pdec
}  // namespace mala
