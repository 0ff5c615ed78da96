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
  int rot, interleaved, G, total, max_new, heads;  // heads: key/value heads of a block
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
// cs[j] = cos and sin of frequencies 2 j and 2 j + 1 of the thread's eight.
__device__ __forceinline__ void rotate(float (&x)[16], const float4 (&cs)[4], int interleaved) {
  auto pair = [](float& a, float& b, float c, float s) {
    const float xa = a, xb = b;
    a = fmaf(xa, c, -xb * s);
    b = fmaf(xb, c, xa * s);
  };
  if (interleaved) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      pair(x[4 * j], x[4 * j + 1], cs[j].x, cs[j].y);
      pair(x[4 * j + 2], x[4 * j + 3], cs[j].z, cs[j].w);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      pair(x[2 * j], x[2 * j + 8], cs[j].x, cs[j].y);
      pair(x[2 * j + 1], x[2 * j + 9], cs[j].z, cs[j].w);
    }
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
// before the first one is rounded and everything is read once; the rotation is done twice
// instead (32 FMA a row and thread, a tenth of the time that the bytes take). LPU and
// PASSES follow the rows that a page can get (host): up to 4 (decode steps): 8 threads, the
// angles in registers; up to 32, 64, 128: one, two, four warps, the angles in shared memory
// for all heads of the block. 4 x 8192 tokens, pages of 128: see the launch.
template <int LPU, int PASSES>
__global__ void __launch_bounds__(APPEND_NT, 2) append_kernel(const AppendParams p) {
  constexpr int UNITS = APPEND_NT / LPU;  // side by side
  constexpr int STEP = LPU / 8;           // rows side by side
  constexpr bool TABLE = LPU > 8;
  extern __shared__ float4 table[];       // [row][4][8]: cs of thread t's j-th pair at [j][t]
  __shared__ float red[APPEND_NT / 32];
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
  const int begin = max(start, slot << p.pool.page_log2);
  const int end = (int)min((long long)len, (long long)(slot + 1) << p.pool.page_log2);
  if (begin >= end) return;
  const int row0 = begin - (slot << p.pool.page_log2), n = end - begin;
  const long long tok0 = (long long)first + (begin - start);
  const int tid = threadIdx.x, t = tid & 7, r0 = (tid % LPU) >> 3;
  const Chunks ch = chunks_of(t, p.rot, p.interleaved);
  const int h0 = blockIdx.z * p.heads, nh = min(p.heads, p.pool.Hkv - h0);
  const int id = page_of(p.pool, b, slot);  // no page: its rows are left out, q is rotated all the same

  if (TABLE && p.rot > 0) {
    const int half = p.rot >> 1;
    for (int e = tid; e < n * (half / 2); e += APPEND_NT) {
      const int r = e / (half / 2), f = 2 * (e - r * (half / 2));
      float4 cs;
      turn(begin + r, p.inv_freq[f], cs.x, cs.y);
      turn(begin + r, p.inv_freq[f + 1], cs.z, cs.w);
      table[r * 32 + ((f >> 1) & 3) * 8 + (f >> 3)] = cs;
    }
    __syncthreads();
  }
  float4 own[TABLE ? 1 : PASSES][4];
  if (!TABLE && ch.freq >= 0) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = make_float2(p.inv_freq[ch.freq + 2 * j], p.inv_freq[ch.freq + 2 * j + 1]);
#pragma unroll
      for (int ps = 0; ps < (TABLE ? 1 : PASSES); ++ps)
        if (ps < n) {
          turn(begin + ps, f.x, own[ps][j].x, own[ps][j].y);
          turn(begin + ps, f.y, own[ps][j].z, own[ps][j].w);
        }
    }
  }
  auto angles = [&](int ps, int r, float4 (&cs)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) cs[j] = TABLE ? table[r * 32 + j * 8 + t] : own[TABLE ? 0 : ps][j];
  };

  const int total = nh * (2 + p.G);  // K of every head, V of every head, Q
  for (int u0 = 0; u0 < total; u0 += UNITS) {
    const int u = u0 + tid / LPU;
    const bool live = u < total;
    const int kind = u < nh ? 0 : (u < 2 * nh ? 1 : 2);
    const bool rotates = kind != 1 && ch.freq >= 0;
    const __nv_bfloat16* src = p.k + (h0 + u) * p.k_head + tok0 * p.k_tok;
    long long stride = p.k_tok;
    if (kind == 1) {
      src = p.v + (h0 + u - nh) * p.v_head + tok0 * p.v_tok;
      stride = p.v_tok;
    } else if (kind == 2) {
      src = p.q + ((long long)h0 * p.G + (u - 2 * nh)) * p.q_head + tok0 * p.q_tok;
      stride = p.q_tok;
    }
    uint4 raw[PASSES][2];
#pragma unroll
    for (int ps = 0; ps < PASSES; ++ps) {
      const int r = r0 + STEP * ps;
      raw[ps][0] = raw[ps][1] = make_uint4(0, 0, 0, 0);
      if (live && r < n && (kind == 2 || id >= 0)) {
        raw[ps][0] = *reinterpret_cast<const uint4*>(src + r * stride + ch.c0);
        raw[ps][1] = *reinterpret_cast<const uint4*>(src + r * stride + ch.c1);
      }
    }
    const bool kv = live && kind < 2 && id >= 0;
    const int h = h0 + (kind == 0 ? u : u - nh);
    uint8_t* base = kind == 0 ? p.pool.k + id * p.pool.k_page + h * p.pool.k_head
                              : p.pool.v + id * p.pool.v_page + h * p.pool.v_head;
    const long long tok = kind == 0 ? p.pool.k_tok : p.pool.v_tok;
    float* scale = (kind == 0 ? p.pool.k_scale : p.pool.v_scale) + (long long)id * p.pool.Hkv + h;
    const float old = kv && row0 > 0 ? *scale : 0.f;  // read by all before it is written below
    float amax = 0.f;
    if (kv) {
#pragma unroll
      for (int ps = 0; ps < PASSES; ++ps) {
        if (r0 + STEP * ps >= n) continue;
        float x[16];
        unpack8(raw[ps][0], x);
        unpack8(raw[ps][1], x + 8);
        if (rotates) {
          float4 cs[4];
          angles(ps, r0 + STEP * ps, cs);
          rotate(x, cs, p.interleaved);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float a = fabsf(x[i]);
          if (a < __int_as_float(0x7f800000)) amax = fmaxf(amax, a);
        }
      }
    }
#pragma unroll
    for (int d = 1; d < (LPU < 32 ? LPU : 32); d <<= 1)
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
    if (LPU > 32) {
      __syncthreads();
      if ((tid & 31) == 0) red[tid >> 5] = amax;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < LPU / 32; ++w) amax = fmaxf(amax, red[(tid / LPU) * (LPU / 32) + w]);
    }
    float s = pow2_scale(amax), ratio = 0.f;
    bool grown = false;
    if (kv && row0 > 0) {
      if (old >= s) {
        s = old;
      } else {
        grown = true;
        ratio = old / s;
      }
    }
    if (kv && tid % LPU == 0) *scale = s;
    if (LPU >= 32) {
      if (grown)
        for (int e = tid % LPU; e < row0 * 8; e += LPU) rescale16(base + (e >> 3) * tok + (e & 7) * 16, ratio);
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
    __nv_bfloat16* dst = p.q_out + ((long long)h0 * p.G + (u - 2 * nh)) * p.qo_head + tok0 * p.qo_tok;
#pragma unroll
    for (int ps = 0; ps < PASSES; ++ps) {
      const int r = r0 + STEP * ps;
      if (!live || r >= n) continue;
      if (kind == 2 && ch.freq < 0) {  // bit for bit
        *reinterpret_cast<uint4*>(dst + r * p.qo_tok + ch.c0) = raw[ps][0];
        *reinterpret_cast<uint4*>(dst + r * p.qo_tok + ch.c1) = raw[ps][1];
        continue;
      }
      float x[16];
      unpack8(raw[ps][0], x);
      unpack8(raw[ps][1], x + 8);
      if (rotates) {
        float4 cs[4];
        angles(ps, r, cs);
        rotate(x, cs, p.interleaved);
      }
      if (kind == 2) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const __nv_bfloat162 z = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
          w[i] = *reinterpret_cast<const uint32_t*>(&z);
        }
        *reinterpret_cast<uint4*>(dst + r * p.qo_tok + ch.c0) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4*>(dst + r * p.qo_tok + ch.c1) = make_uint4(w[4], w[5], w[6], w[7]);
      } else if (kv) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 16; ++i)  // e4m3 has no infinities
          if (!(fabsf(x[i]) < __int_as_float(0x7f800000))) x[i] = __int_as_float(0x7fc00000);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = floats_to_e4m3x2(x[4 * i] * inv, x[4 * i + 1] * inv) |
                 floats_to_e4m3x2(x[4 * i + 2] * inv, x[4 * i + 3] * inv) << 16;
        uint8_t* row = base + (row0 + r) * tok;
        *reinterpret_cast<uint2*>(row + ch.c0) = make_uint2(w[0], w[1]);
        *reinterpret_cast<uint2*>(row + ch.c1) = make_uint2(w[2], w[3]);
      }
    }
  }
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
