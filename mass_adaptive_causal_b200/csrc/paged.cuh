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
//    earlier tokens are re-rounded without loss (but for values that fall among
//    e4m3's subnormals: an error of at most 2^-10 of the new scale);
//  - the cache's content does not depend on how its tokens came in;
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
  int rot, interleaved, G, total, max_new;
};

constexpr int APPEND_NT = 256;

__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// A thread holds sixteen of a row's 128 values: two chunks of eight, c0 and
// c1, chosen so that every rotated pair lies within the thread.
struct Chunks {
  int c0, c1;   // first dimension of each chunk
  int freq;     // index of the first of its eight frequencies, -1: not rotated
};
__device__ __forceinline__ Chunks chunks_of(int t, int rot, int interleaved) {
  Chunks c;
  const int pairs = rot >> 4;  // threads that rotate
  c.freq = t < pairs ? 8 * t : -1;
  if (interleaved || t >= pairs) {  // (x_2i, x_2i+1), or the part that is not rotated
    c.c0 = 16 * t;
    c.c1 = 16 * t + 8;
  } else {  // (x_i, x_{i + rot/2})
    c.c0 = 8 * t;
    c.c1 = 8 * t + (rot >> 1);
  }
  return c;
}
__device__ __forceinline__ void rotate(float (&x)[16], const float (&cs)[8], const float (&sn)[8],
                                       int interleaved) {
  auto pair = [](float& a, float& b, float c, float s) {
    const float xa = a, xb = b;
    a = fmaf(xa, c, -xb * s);
    b = fmaf(xb, c, xa * s);
  };
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) pair(x[2 * i], x[2 * i + 1], cs[i], sn[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) pair(x[i], x[i + 8], cs[i], sn[i]);
  }
}

__device__ __forceinline__ float block_max(float x, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  x = red[0];
#pragma unroll
  for (int w = 1; w < APPEND_NT / 32; ++w) x = fmaxf(x, red[w]);
  return x;
}

// Writes the rows [row0, row0 + n) of one page and head, whose values this
// block's threads hold (x[pass], rows `tid / 8 + 32 * pass`), and settles the
// page's scale. The rows below row0 hold earlier tokens.
template <int PASSES>
__device__ __forceinline__ void store_page(uint8_t* base, long long tok, float* scale, int row0,
                                           int n, const Chunks& ch, float (&x)[PASSES][16],
                                           float* red) {
  const int r0 = threadIdx.x >> 3;
  float amax = 0.f;
#pragma unroll
  for (int p = 0; p < PASSES; ++p)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float a = fabsf(x[p][i]);
      if (a < __int_as_float(0x7f800000)) amax = fmaxf(amax, a);
      else x[p][i] = __int_as_float(0x7fc00000);  // e4m3 has no infinities
    }
  amax = block_max(amax, red);
  float s = pow2_scale(amax);
  if (row0 > 0) {
    const float old = *scale;
    if (old >= s) {
      s = old;
    } else {
      const float ratio = old / s;
      for (int e = threadIdx.x; e < row0 * 8; e += APPEND_NT) {
        uint4* at = reinterpret_cast<uint4*>(base + (e >> 3) * tok + (e & 7) * 16);
        uint4 u = *at;
        uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 lo = f16x2_to_float2(e4m3x2_to_f16x2(w[i]));
          const float2 hi = f16x2_to_float2(e4m3x2_hi_to_f16x2(w[i]));
          w[i] = floats_to_e4m3x2(lo.x * ratio, lo.y * ratio) |
                 floats_to_e4m3x2(hi.x * ratio, hi.y * ratio) << 16;
        }
        *at = u;
      }
    }
    __syncthreads();  // every thread has read the old scale
  }
  if (threadIdx.x == 0) *scale = s;
  const float inv = 1.f / s;
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const int r = r0 + 32 * p;
    if (r >= n) continue;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = floats_to_e4m3x2(x[p][4 * i] * inv, x[p][4 * i + 1] * inv) |
             floats_to_e4m3x2(x[p][4 * i + 2] * inv, x[p][4 * i + 3] * inv) << 16;
    uint8_t* row = base + (row0 + r) * tok;
    *reinterpret_cast<uint2*>(row + ch.c0) = make_uint2(w[0], w[1]);
    *reinterpret_cast<uint2*>(row + ch.c1) = make_uint2(w[2], w[3]);
  }
}

// One block per (page of new tokens, sequence, key/value head): rotates and
// stores the page's new K and V rows and rotates the head's G query heads.
template <int PASSES>
__global__ void __launch_bounds__(APPEND_NT) append_kernel(const AppendParams p) {
  __shared__ float red[APPEND_NT / 32];
  const int b = blockIdx.y, h = blockIdx.z;
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
  const int page = p.pool.page;
  const int slot = start / page + blockIdx.x;
  const int begin = max(start, slot * page), end = min(len, (slot + 1) * page);
  if (begin >= end) return;
  const int row0 = begin - slot * page, n = end - begin;
  const int t = threadIdx.x & 7, r0 = threadIdx.x >> 3;
  const Chunks ch = chunks_of(t, p.rot, p.interleaved);
  const long long tok0 = (long long)first + (begin - start);

  float freq[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) freq[i] = ch.freq >= 0 ? p.inv_freq[ch.freq + i] : 0.f;
  float x[PASSES][16];
#pragma unroll
  for (int ps = 0; ps < PASSES; ++ps) {
    const int r = r0 + 32 * ps;
#pragma unroll
    for (int i = 0; i < 16; ++i) x[ps][i] = 0.f;
    if (r >= n) continue;
    const __nv_bfloat16* row = p.k + (tok0 + r) * p.k_tok + h * p.k_head;
    float lo[8], hi[8];
    unpack8(*reinterpret_cast<const uint4*>(row + ch.c0), lo);
    unpack8(*reinterpret_cast<const uint4*>(row + ch.c1), hi);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[ps][i] = lo[i];
      x[ps][8 + i] = hi[i];
    }
    float cs[8], sn[8];
    if (ch.freq >= 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) turn(begin + r, freq[i], cs[i], sn[i]);
      rotate(x[ps], cs, sn, p.interleaved);
    }
    if (p.q) {
      for (int g = 0; g < p.G; ++g) {
        const int hq = h * p.G + g;
        const __nv_bfloat16* qr = p.q + (tok0 + r) * p.q_tok + hq * p.q_head;
        __nv_bfloat16* qo = p.q_out + (tok0 + r) * p.qo_tok + hq * p.qo_head;
        const uint4 u0 = *reinterpret_cast<const uint4*>(qr + ch.c0);
        const uint4 u1 = *reinterpret_cast<const uint4*>(qr + ch.c1);
        if (ch.freq < 0) {
          *reinterpret_cast<uint4*>(qo + ch.c0) = u0;
          *reinterpret_cast<uint4*>(qo + ch.c1) = u1;
          continue;
        }
        float y[16];
        unpack8(u0, lo);
        unpack8(u1, hi);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          y[i] = lo[i];
          y[8 + i] = hi[i];
        }
        rotate(y, cs, sn, p.interleaved);
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const __nv_bfloat162 z = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
          w[i] = *reinterpret_cast<const uint32_t*>(&z);
        }
        *reinterpret_cast<uint4*>(qo + ch.c0) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4*>(qo + ch.c1) = make_uint4(w[4], w[5], w[6], w[7]);
      }
    }
  }
  const int id = page_of(p.pool, b, slot);
  if (id < 0) return;
  store_page<PASSES>(p.pool.k + id * p.pool.k_page + h * p.pool.k_head, p.pool.k_tok,
                     p.pool.k_scale + (long long)id * p.pool.Hkv + h, row0, n, ch, x, red);
#pragma unroll
  for (int ps = 0; ps < PASSES; ++ps) {
    const int r = r0 + 32 * ps;
#pragma unroll
    for (int i = 0; i < 16; ++i) x[ps][i] = 0.f;
    if (r >= n) continue;
    const __nv_bfloat16* row = p.v + (tok0 + r) * p.v_tok + h * p.v_head;
    float lo[8], hi[8];
    unpack8(*reinterpret_cast<const uint4*>(row + ch.c0), lo);
    unpack8(*reinterpret_cast<const uint4*>(row + ch.c1), hi);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[ps][i] = lo[i];
      x[ps][8 + i] = hi[i];
    }
  }
  store_page<PASSES>(p.pool.v + id * p.pool.v_page + h * p.pool.v_head, p.pool.v_tok,
                     p.pool.v_scale + (long long)id * p.pool.Hkv + h, row0, n, ch, x, red);
}

struct GatherParams {
  Pool pool;
  const int32_t* cu;  // [batch + 1]
  __nv_bfloat16* k;   // [total][Hkv][128]
  __nv_bfloat16* v;
  int total, max_seqlen;
};

constexpr int GATHER_NT = 256;

__device__ __forceinline__ uint4 dequant8(uint32_t a, uint32_t b, float s) {
  const uint32_t in[2] = {a, b};
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

// One block per (page, sequence): every head's K and V rows of the page.
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
  const int per_head = n * 8;  // 16-value chunks
  for (int e = threadIdx.x; e < Hkv * per_head; e += GATHER_NT) {
    const int h = e / per_head, rest = e - h * per_head;
    const int r = rest >> 3, c = (rest & 7) * 16;
    const long long out = (((long long)first + begin + r) * Hkv + h) * D + c;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const uint8_t* src = w ? p.pool.v + id * p.pool.v_page + h * p.pool.v_head + r * p.pool.v_tok
                             : p.pool.k + id * p.pool.k_page + h * p.pool.k_head + r * p.pool.k_tok;
      __nv_bfloat16* dst = (w ? p.v : p.k) + out;
      uint4 u = make_uint4(0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu);  // NaN
      float s = 1.f;
      if (id >= 0) {
        u = *reinterpret_cast<const uint4*>(src + c);
        s = (w ? p.pool.v_scale : p.pool.k_scale)[(long long)id * Hkv + h];
      }
      *reinterpret_cast<uint4*>(dst) = dequant8(u.x, u.y, s);
      *reinterpret_cast<uint4*>(dst + 8) = dequant8(u.z, u.w, s);
    }
  }
}

}  // namespace paged
}  // namespace mala
