// paged.cuh -- the paged key/value cache in 8 bits: its view in device code,
// the appending of new tokens (with the rotation by position on the way) and
// the reading back as packed bf16. The decode step over it is in
// decode_paged_sm100.cuh.
//
// Pages hold e4m3 values [Hkv][page][128] and one float32 scale per page and
// key/value head; a value is e4m3 * scale. Appending writes scales that are
// powers of two: e4m3 is itself a floating-point format, so a scale's mantissa
// would buy no precision, while with powers of two
//  - a later, larger token of the page only adds to the exponent, and the
//    earlier tokens are re-rounded without loss, but for values that sink among
//    e4m3's subnormals, 2^-9 of the scale apart: each growth rounds those by at
//    most 2^-10 of the scale it leads to, all growths by less than 2^-9 of the
//    last one (the scales at least double);
//  - so the cache's content does not depend on how its tokens came in, but for
//    such values, which may come out one subnormal step apart;
//  - a dequantized value is exact in bf16.
#pragma once

#include "common.cuh"

namespace mala {
namespace paged {

constexpr int D = 128;
constexpr float kE4m3Max = 448.f;
constexpr int kMinExp = -100;  // the smallest scale is 2^-100

struct Pool {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;  // [num_pages][Hkv]
  float* v_scale;
  const int32_t* table;  // [sequences][max_pages], rows table_stride apart
  long long k_page, k_head, k_tok, v_page, v_head, v_tok;  // strides in bytes
  long long table_stride;
  int num_pages, page, page_log2, max_pages, Hkv;
};

// The page that holds position `pos` of sequence b, or -1 (and a status) when
// the table has no entry for it or the entry is no page of the pool.
__device__ __forceinline__ int page_of(const Pool& p, int b, int slot) {
  int id = -1;
  if (slot < p.max_pages) id = p.table[(long long)b * p.table_stride + slot];
  if (id < 0 || id >= p.num_pages) {
    record_bad_page(0x500);
    return -1;
  }
  return id;
}

// Two e4m3 values (low byte first) as packed halves; exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t h;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
      : "=r"(h)
      : "r"(two));
  return h;
}
__device__ __forceinline__ uint32_t e4m3x2_hi_to_f16x2(uint32_t four) {
  uint32_t h;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}"
      : "=r"(h)
      : "r"(four));
  return h;
}
__device__ __forceinline__ float2 f16x2_to_float2(uint32_t h) {
  const __half2 x = *reinterpret_cast<const __half2*>(&h);
  return __half22float2(x);
}
// a -> low byte, b -> high byte, to nearest even; NaN stays NaN.
__device__ __forceinline__ uint32_t floats_to_e4m3x2(float a, float b) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

// The least power of two s >= 2^kMinExp with amax <= 448 s; 448 = 1.75 * 2^8,
// so s follows from amax's exponent and whether its mantissa is above 1.75.
// A subnormal amax is far below the least scale's range.
__device__ __forceinline__ float pow2_scale(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = e < kMinExp ? kMinExp : e;
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// cos and sin of 2 pi x for the angle's number of turns x = pos * inv_freq /
// (2 pi), reduced in float64 (a float32 product loses the angle of a far
// position: at 131072 rad it is off by up to 0.008). The reduced angle
// goes through sincospif as a float32 plus the rest it leaves, so that both
// values are good to about one float32 step.
__device__ __forceinline__ void turn(int pos, float inv_freq, float& c, float& s) {
  double x = (double)pos * (double)inv_freq * 0.15915494309189535;
  x -= rint(x);
  const double h = 2.0 * x;  // half turns in [-1, 1]
  const float hi = (float)h;
  const float rest = (float)(h - (double)hi) * 3.14159265f;
  float s0, c0;
  sincospif(hi, &s0, &c0);
  c = fmaf(-s0, rest, c0);
  s = fmaf(c0, rest, s0);
}

struct AppendParams {
  Pool pool;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const __nv_bfloat16* q;  // may be null
  __nv_bfloat16* q_out;
  long long k_tok, k_head, v_tok, v_head, q_tok, q_head, qo_tok, qo_head;  // elements
  const int32_t* cu;        // [batch + 1] or null: one new token per sequence
  const int32_t* seq_lens;  // [batch], new tokens included
  const float* inv_freq;    // [rot / 2]
  int rot, G, total, max_new, heads;  // heads: key/value heads of a block
};

constexpr int APPEND_NT = 256;

__device__ __forceinline__ void unpack8(const uint4& u, float* x) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// A thread holds sixteen of a row's 128 values: two chunks of eight, c0 and
// c1, chosen so that every rotated pair lies within the thread and that neighbours' chunks lie
// side by side (a store then fills whole sectors): of the rotated part the t-th chunk of
// each half, of the rest likewise. Pairs (x_i, x_{i + rot/2}) have their elements in c0 and
// c1, pairs (x_2i, x_2i+1) both in one.
struct Chunks {
  int c0, c1;   // first dimension of each chunk
  bool rotated;
};
__device__ __forceinline__ Chunks chunks_of(int t, int rot) {
  Chunks c;
  const int pairs = rot >> 4;  // threads that rotate
  c.rotated = t < pairs;
  c.c0 = c.rotated ? 8 * t : rot + 8 * (t - pairs);
  c.c1 = c.c0 + ((c.rotated ? rot : 128 - rot) >> 1);
  return c;
}
// The thread's k-th frequency (of eight), and whose f is and which.
template <bool INTERLEAVED>
__device__ __forceinline__ int freq_of(int t, int k, int rot) {
  if (!INTERLEAVED) return 8 * t + k;
  return 4 * t + (k < 4 ? k : (rot >> 2) + k - 4);
}
template <bool INTERLEAVED>
__device__ __forceinline__ int freq_slot(int f, int rot) {  // 8 t + k
  if (!INTERLEAVED) return f;
  const int half = f >= rot >> 2 ? 1 : 0, g = f - half * (rot >> 2);
  return 8 * (g >> 2) + 4 * half + (g & 3);
}

// Two floats side by side, and the two-at-a-time instructions on them.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 split2(f32x2 x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// cs[j] = cos, cos, sin, sin of the thread's frequencies 2 j and 2 j + 1. Each result is a
// product rounded and a sum of products rounded once.
template <bool INTERLEAVED>
__device__ __forceinline__ void rotate(float (&x)[16], const float4 (&cs)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const f32x2 c = pack2(cs[j].x, cs[j].y), s = pack2(cs[j].z, cs[j].w);
    const f32x2 minus = mul2(s, pack2(-1.f, -1.f));
    // the pairs' first and second elements
    constexpr int A = INTERLEAVED ? 4 : 2, STEP = INTERLEAVED ? 2 : 1, B = INTERLEAVED ? 1 : 8;
    const f32x2 a = pack2(x[A * j], x[A * j + STEP]);
    const f32x2 b = pack2(x[A * j + B], x[A * j + STEP + B]);
    const float2 ra = split2(fma2(b, minus, mul2(a, c)));
    const float2 rb = split2(fma2(a, s, mul2(b, c)));
    x[A * j] = ra.x;
    x[A * j + STEP] = ra.y;
    x[A * j + B] = rb.x;
    x[A * j + STEP + B] = rb.y;
  }
}

// Sixteen e4m3 values that lay under another scale: times ratio, rounded again.
__device__ __forceinline__ void rescale16(uint8_t* p, float ratio) {
  uint4 u = *reinterpret_cast<const uint4*>(p);
  uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 lo = f16x2_to_float2(e4m3x2_to_f16x2(w[i]));
    const float2 hi = f16x2_to_float2(e4m3x2_hi_to_f16x2(w[i]));
    w[i] = floats_to_e4m3x2(lo.x * ratio, lo.y * ratio) |
           floats_to_e4m3x2(hi.x * ratio, hi.y * ratio) << 16;
  }
  *reinterpret_cast<uint4*>(p) = u;
}

// One block per (page of new tokens, sequence, group of key/value heads). Its units are the
// new rows of one head: K and V (rotate, find the page's scale, round, store) and Q
// (rotate, store). A unit is LPU threads' work, eight of them a row, each thread holding
// PASSES rows' sixteen values as they were loaded, so that a page's largest value is known
// before the first one is rounded and everything is read once; K is rotated twice instead. As
// soon as a row is stored, the next unit's takes its registers, so loads are always under way.
// LPU and PASSES follow the rows that a page can get (host): up to 2 (decode steps): 8 threads,
// the angles in registers; up to 32, 64, 128: one, two, four warps, the angles in shared
// memory for all heads of the block. 4 x 8192 tokens of 8 + 32 heads, pages of 128: 143 us (5.2 TB/s,
// 79% of the measured copy bandwidth; 48% of the issue slots with sixteen warps an SM, without
// rotation 124 us). Four rows a thread and 256 threads a unit, three blocks to an SM instead of
// two: 183 us. 256 single tokens: 7.7 us, latency (where no scale grows; 16 us where 40% do, their
// earlier rows read and written by a warp for its four units in turn).
template <int LPU, int PASSES, bool INTERLEAVED>
__global__ void __launch_bounds__(APPEND_NT, 2) append_kernel(const AppendParams p) {
  constexpr int UNITS = APPEND_NT / LPU;  // side by side
  constexpr int STEP = LPU / 8;           // rows side by side
  constexpr bool TABLE = LPU > 8;
  extern __shared__ float4 table[];       // [row][4][8]: cs[j] of thread t at [j][t]
  __shared__ float red[APPEND_NT / 32];
  const float inf = __int_as_float(0x7f800000);
  const int b = blockIdx.y;
  int first = b, count = 1;
  if (p.cu) {
    first = p.cu[b];
    count = p.cu[b + 1] - first;
  }
  const int len = p.seq_lens[b];
  if (count <= 0 || len <= 0) return;  // nothing new, or an unused slot of the batch
  if (len < count || count > p.max_new || first < 0 || first > p.total - count) {
    if (threadIdx.x == 0) record_bad_page(0x501);
    return;
  }
  const int start = len - count;
  const int slot = (start >> p.pool.page_log2) + blockIdx.x;
  if ((long long)slot << p.pool.page_log2 >= len) return;
  const int begin = max(start, slot << p.pool.page_log2);
  const int end = (int)min((long long)len, (long long)(slot + 1) << p.pool.page_log2);
  const int row0 = begin - (slot << p.pool.page_log2), n = end - begin;
  const long long tok0 = (long long)first + (begin - start);
  const int tid = threadIdx.x, t = tid & 7, r0 = (tid % LPU) >> 3;
  const Chunks ch = chunks_of(t, p.rot);
  const int h0 = blockIdx.z * p.heads, nh = min(p.heads, p.pool.Hkv - h0);
  const int id = page_of(p.pool, b, slot);  // no page: its rows are left out, q is rotated all the same

  // the units: K of every head, V of every head, Q. With the angles in a table Q is not cut into
  // units but walked along the tokens, all heads of one side by side, as it lies in memory.
  const int nq = nh * p.G;
  const int total = 2 * nh + (TABLE ? 0 : nq);
  const __nv_bfloat16* src = nullptr;
  long long stride = 0;
  auto aim = [&](int u) {
    if (u < nh) {
      src = p.k + (h0 + u) * p.k_head + tok0 * p.k_tok;
      stride = p.k_tok;
    } else if (u < 2 * nh) {
      src = p.v + (h0 + u - nh) * p.v_head + tok0 * p.v_tok;
      stride = p.v_tok;
    } else {
      src = p.q + ((long long)h0 * p.G + (u - 2 * nh)) * p.q_head + tok0 * p.q_tok;
      stride = p.q_tok;
    }
  };
  uint4 raw[PASSES][2];
  auto load = [&](int ps, bool live) {
    const int r = r0 + STEP * ps;
    if (live && r < n) {
      raw[ps][0] = *reinterpret_cast<const uint4*>(src + r * stride + ch.c0);
      raw[ps][1] = *reinterpret_cast<const uint4*>(src + r * stride + ch.c1);
    }
  };
  // Q's rows and heads, the next to be loaded (lq) and to be stored (sq)
  struct At {
    int row, head;
  } lq = {0, 0}, sq;
  if (TABLE && nq > 0) {
    lq.row = (tid >> 3) / nq;
    lq.head = (tid >> 3) - lq.row * nq;
  } else {
    lq.row = n;  // none
  }
  sq = lq;
  const int q_rows = nq > 0 ? (APPEND_NT / 8) / nq : 0, q_heads = APPEND_NT / 8 - q_rows * nq;
  auto step = [&](At& a) {
    a.row += q_rows;
    a.head += q_heads;
    if (a.head >= nq) {
      a.head -= nq;
      ++a.row;
    }
  };
  auto load_q = [&](int ps) {
    if (lq.row >= n) return;
    const __nv_bfloat16* at = p.q + (tok0 + lq.row) * p.q_tok +
                              ((long long)h0 * p.G + lq.head) * p.q_head;
    raw[ps][0] = *reinterpret_cast<const uint4*>(at + ch.c0);
    raw[ps][1] = *reinterpret_cast<const uint4*>(at + ch.c1);
    step(lq);
  };
  aim(tid / LPU);
#pragma unroll
  for (int ps = 0; ps < PASSES; ++ps) {
    if (tid / LPU < total)
      load(ps, true);
    else if (TABLE)
      load_q(ps);
  }

  if (TABLE && p.rot > 0) {
    const int quarter = p.rot >> 2;
    for (int e = tid; e < n * quarter; e += APPEND_NT) {
      const int r = e / quarter, f = 2 * (e - r * quarter);
      float4 cs;
      turn(begin + r, p.inv_freq[f], cs.x, cs.z);
      turn(begin + r, p.inv_freq[f + 1], cs.y, cs.w);
      const int k = freq_slot<INTERLEAVED>(f, p.rot);
      table[r * 32 + ((k >> 1) & 3) * 8 + (k >> 3)] = cs;
    }
    __syncthreads();
  }
  float4 own[TABLE ? 1 : PASSES][4];
  if (!TABLE && ch.rotated) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = make_float2(p.inv_freq[freq_of<INTERLEAVED>(t, 2 * j, p.rot)],
                                   p.inv_freq[freq_of<INTERLEAVED>(t, 2 * j + 1, p.rot)]);
#pragma unroll
      for (int ps = 0; ps < (TABLE ? 1 : PASSES); ++ps)
        if (ps < n) {
          turn(begin + ps, f.x, own[ps][j].x, own[ps][j].z);
          turn(begin + ps, f.y, own[ps][j].y, own[ps][j].w);
        }
    }
  }
  // a row's values in float32, rotated
  auto values = [&](int ps, int r, bool rotates, float (&x)[16]) {
    unpack8(raw[ps][0], x);
    unpack8(raw[ps][1], x + 8);
    if (!rotates) return;
    float4 cs[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      cs[j] = TABLE ? table[r * 32 + j * 8 + t] : own[TABLE ? 0 : ps][j];
    rotate<INTERLEAVED>(x, cs);
  };
  auto store_q = [&](int ps, int r, __nv_bfloat16* dst) {
    uint4 w[2] = {raw[ps][0], raw[ps][1]};  // not rotated: bit for bit
    if (ch.rotated) {
      float x[16];
      values(ps, r, true, x);
      uint32_t* z = reinterpret_cast<uint32_t*>(w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const __nv_bfloat162 y = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        z[i] = *reinterpret_cast<const uint32_t*>(&y);
      }
    }
    *reinterpret_cast<uint4*>(dst + ch.c0) = w[0];
    *reinterpret_cast<uint4*>(dst + ch.c1) = w[1];
  };

  for (int u0 = 0; u0 < total; u0 += UNITS) {
    const int u = u0 + tid / LPU;
    const bool more = u + UNITS < total;
    aim(u + UNITS);
    const bool kv = u < 2 * nh, keys = u < nh;
    const bool rotates = (keys || !kv) && ch.rotated;
    if (u0 < 2 * nh) {  // some of the block's units are K or V
      const bool store = kv && id >= 0;
      const int h = h0 + (keys ? u : u - nh);
      uint8_t* base = keys ? p.pool.k + id * p.pool.k_page + h * p.pool.k_head
                           : p.pool.v + id * p.pool.v_page + h * p.pool.v_head;
      const long long tok = keys ? p.pool.k_tok : p.pool.v_tok;
      float* scale = (keys ? p.pool.k_scale : p.pool.v_scale) + (long long)id * p.pool.Hkv + h;
      const float old = store && row0 > 0 ? *scale : 0.f;  // read by all before it is written below
      auto largest = [&](bool finite) {
        float m = 0.f;
        if (store) {
#pragma unroll
          for (int ps = 0; ps < PASSES; ++ps) {
            if (r0 + STEP * ps >= n) continue;
            float x[16];
            values(ps, r0 + STEP * ps, rotates, x);
#pragma unroll
            for (int i = 0; i < 16; ++i)  // a NaN is passed over
              m = fmaxf(m, finite && fabsf(x[i]) == inf ? 0.f : fabsf(x[i]));
          }
        }
#pragma unroll
        for (int d = 1; d < (LPU < 32 ? LPU : 32); d <<= 1)
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        if (LPU > 32) {
          __syncthreads();
          if ((tid & 31) == 0) red[tid >> 5] = m;
          __syncthreads();
#pragma unroll
          for (int w = 0; w < LPU / 32; ++w) m = fmaxf(m, red[(tid / LPU) * (LPU / 32) + w]);
        }
        return m;
      };
      float amax = largest(false);
      const bool infinite = amax == inf;
      // once more without the infinities, where there are any
      if (LPU > 32 ? __syncthreads_or(infinite) : __any_sync(0xffffffffu, infinite))
        amax = largest(true);
      float s = pow2_scale(amax), ratio = 0.f;
      bool grown = false;
      if (store && row0 > 0) {
        if (old >= s) {
          s = old;
        } else {
          grown = true;
          ratio = old / s;
        }
      }
      if (store && tid % LPU == 0) *scale = s;
      if (LPU >= 32) {
        if (grown)
#pragma unroll 4
          for (int e = tid % LPU; e < row0 * 8; e += LPU)
            rescale16(base + (e >> 3) * tok + (e & 7) * 16, ratio);
      } else {  // the whole warp, one of its units after the other
        uint32_t todo = __ballot_sync(0xffffffffu, grown && tid % LPU == 0);
        while (todo) {
          const int lane = __ffs(todo) - 1;
          todo &= todo - 1;
          const unsigned long long at =
              __shfl_sync(0xffffffffu, (unsigned long long)(uintptr_t)base, lane);
          const long long step = __shfl_sync(0xffffffffu, tok, lane);
          const float by = __shfl_sync(0xffffffffu, ratio, lane);
#pragma unroll 4
          for (int e = tid & 31; e < row0 * 8; e += 32)
            rescale16(reinterpret_cast<uint8_t*>((uintptr_t)at) + (e >> 3) * step + (e & 7) * 16, by);
        }
      }
      const float inv = 1.f / s;
      if (kv) {
#pragma unroll
        for (int ps = 0; ps < PASSES; ++ps) {
          const int r = r0 + STEP * ps;
          if (r < n && id >= 0) {
            float x[16];
            values(ps, r, rotates, x);
            if (infinite)  // e4m3 has none
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (fabsf(x[i]) == inf) x[i] = __int_as_float(0x7fc00000);
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[i] = floats_to_e4m3x2(x[4 * i] * inv, x[4 * i + 1] * inv) |
                     floats_to_e4m3x2(x[4 * i + 2] * inv, x[4 * i + 3] * inv) << 16;
            uint8_t* row = base + (row0 + r) * tok;
            *reinterpret_cast<uint2*>(row + ch.c0) = make_uint2(w[0], w[1]);
            *reinterpret_cast<uint2*>(row + ch.c1) = make_uint2(w[2], w[3]);
          }
          if (TABLE && !more)
            load_q(ps);
          else
            load(ps, more);
        }
      }
    }
    if (!TABLE && !kv && u < total) {
      __nv_bfloat16* dst = p.q_out + ((long long)h0 * p.G + (u - 2 * nh)) * p.qo_head + tok0 * p.qo_tok;
#pragma unroll
      for (int ps = 0; ps < PASSES; ++ps) {
        const int r = r0 + STEP * ps;
        if (r < n) store_q(ps, r, dst + r * p.qo_tok);
        load(ps, more);
      }
    }
  }
  if (TABLE)
    while (sq.row < n) {
#pragma unroll
      for (int ps = 0; ps < PASSES; ++ps) {
        if (sq.row >= n) break;
        store_q(ps, sq.row, p.q_out + (tok0 + sq.row) * p.qo_tok +
                                ((long long)h0 * p.G + sq.head) * p.qo_head);
        step(sq);
        load_q(ps);
      }
    }
}

using AppendKernel = void (*)(AppendParams);
inline AppendKernel append_kernel_of(int rows, bool interleaved) {
  if (rows <= 2) return interleaved ? append_kernel<8, 2, true> : append_kernel<8, 2, false>;
  if (rows <= 32) return interleaved ? append_kernel<32, 8, true> : append_kernel<32, 8, false>;
  if (rows <= 64) return interleaved ? append_kernel<64, 8, true> : append_kernel<64, 8, false>;
  return interleaved ? append_kernel<128, 8, true> : append_kernel<128, 8, false>;
}

struct GatherParams {
  Pool pool;
  const int32_t* cu;  // [batch + 1]
  __nv_bfloat16* k;   // [total][Hkv][128]
  __nv_bfloat16* v;
  int total, max_seqlen;
};

constexpr int GATHER_NT = 256;

__device__ __forceinline__ uint4 dequant8(const uint2& u, float s) {
  const uint32_t in[2] = {u.x, u.y};
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 lo = f16x2_to_float2(e4m3x2_to_f16x2(in[i]));
    const float2 hi = f16x2_to_float2(e4m3x2_hi_to_f16x2(in[i]));
    const __nv_bfloat162 z0 = __floats2bfloat162_rn(lo.x * s, lo.y * s);
    const __nv_bfloat162 z1 = __floats2bfloat162_rn(hi.x * s, hi.y * s);
    w[2 * i] = *reinterpret_cast<const uint32_t*>(&z0);
    w[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&z1);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// One block per (page, sequence): every head's K and V rows of the page, eight values a thread, so
// that a warp writes 512 bytes in a row. 4 x 131072 tokens of 8 heads (1.07 GB read, 2.15 GB
// written): 555 us, 88% of the measured copy bandwidth, the same with more loads under way.
__global__ void __launch_bounds__(GATHER_NT) gather_kernel(const GatherParams p) {
  const int b = blockIdx.y, slot = blockIdx.x;
  const int first = p.cu[b], len = p.cu[b + 1] - first;
  if (len <= 0) return;
  if (len > p.max_seqlen || first < 0 || first > p.total - len) {
    if (threadIdx.x == 0) record_bad_page(0x502);
    return;
  }
  const int page = p.pool.page, Hkv = p.pool.Hkv;
  const int begin = slot * page, n = min(len - begin, page);
  if (n <= 0) return;
  const int id = page_of(p.pool, b, slot);
  const int per_head = n * 16;  // eight values each
  for (int e = threadIdx.x; e < Hkv * per_head; e += GATHER_NT) {
    const int h = e / per_head, rest = e - h * per_head;
    const int r = rest >> 4, c = (rest & 15) * 8;
    const long long out = (((long long)first + begin + r) * Hkv + h) * D + c;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const uint8_t* src = w ? p.pool.v + id * p.pool.v_page + h * p.pool.v_head + r * p.pool.v_tok
                             : p.pool.k + id * p.pool.k_page + h * p.pool.k_head + r * p.pool.k_tok;
      __nv_bfloat16* dst = (w ? p.v : p.k) + out;
      uint2 u = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);  // NaN
      float s = 1.f;
      if (id >= 0) {
        u = *reinterpret_cast<const uint2*>(src + c);
        s = (w ? p.pool.v_scale : p.pool.k_scale)[(long long)id * Hkv + h];
      }
      *reinterpret_cast<uint4*>(dst) = dequant8(u, s);
    }
  }
}

}  // namespace paged
}  // namespace mala
