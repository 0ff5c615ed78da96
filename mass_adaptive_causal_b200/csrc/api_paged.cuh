// api_paged.cuh -- the C entry points of the paged 8-bit cache: argument
// checks and launches (the contract is in include/mala.h).
#pragma once

#include <atomic>

#include "api.cuh"
#include "decode_paged_sm100.cuh"
#include "paged.cuh"

namespace mala {
namespace host {

constexpr long long kMaxPositions = 0x7fffffffll - 256;

// Checks the cache's description and turns it into the kernels' view.
inline mala_status make_pool(const mala_paged_cache* c, paged::Pool* p) {
  if (!c) return MALA_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->max_pages < 1 || c->Hkv < 1 || c->Hkv > 65535)
    return MALA_ERR_INVALID_ARG;
  if (c->d != paged::D || (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 &&
                           c->page_size != 128))
    return MALA_ERR_UNSUPPORTED;
  if ((long long)c->max_pages * c->page_size > kMaxPositions) return MALA_ERR_INVALID_ARG;
  if (!c->k_pages || !c->v_pages || !c->k_scale || !c->v_scale || !c->page_table)
    return MALA_ERR_INVALID_ARG;
  if (!aligned16(c->k_pages) || !aligned16(c->v_pages)) return MALA_ERR_INVALID_ARG;
  const void* words[] = {c->k_scale, c->v_scale, c->page_table};
  for (const void* w : words)
    if (reinterpret_cast<uintptr_t>(w) & 3u) return MALA_ERR_INVALID_ARG;
  const int64_t strides[] = {c->k_stride_page, c->k_stride_head, c->k_stride_token,
                             c->v_stride_page, c->v_stride_head, c->v_stride_token};
  const int extent[] = {c->num_pages, c->Hkv, c->page_size};
  for (int i = 0; i < 6; ++i)
    if (extent[i % 3] > 1 &&
        (strides[i] < paged::D || (strides[i] & 15) || strides[i] >= (1ll << 40)))
      return MALA_ERR_INVALID_ARG;
  if (c->table_stride < c->max_pages) return MALA_ERR_INVALID_ARG;
  p->k = reinterpret_cast<uint8_t*>(c->k_pages);
  p->v = reinterpret_cast<uint8_t*>(c->v_pages);
  p->k_scale = c->k_scale;
  p->v_scale = c->v_scale;
  p->table = c->page_table;
  p->k_page = c->k_stride_page;
  p->k_head = c->k_stride_head;
  p->k_tok = c->k_stride_token;
  p->v_page = c->v_stride_page;
  p->v_head = c->v_stride_head;
  p->v_tok = c->v_stride_token;
  p->table_stride = c->table_stride;
  p->num_pages = c->num_pages;
  p->page = c->page_size;
  p->page_log2 = c->page_size == 16 ? 4 : c->page_size == 32 ? 5 : c->page_size == 64 ? 6 : 7;
  p->max_pages = c->max_pages;
  p->Hkv = c->Hkv;
  return MALA_OK;
}

// One side of the pool as a 4-D byte tensor (x = d, y = token, z = head, w =
// page), a box of one page and head, 128-byte swizzle.
inline bool make_page_map(CUtensorMap* m, const void* base, const paged::Pool& p, long long page,
                          long long head, long long tok) {
  auto enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[4] = {(cuuint64_t)paged::D, (cuuint64_t)p.page, (cuuint64_t)p.Hkv,
                        (cuuint64_t)p.num_pages};
  // the stride of a dimension of extent 1 is never used, but has to be legal
  cuuint64_t strides[3] = {(cuuint64_t)tok, (cuuint64_t)(p.Hkv > 1 ? head : paged::D),
                           (cuuint64_t)(p.num_pages > 1 ? page : paged::D)};
  cuuint32_t box[4] = {(cuuint32_t)paged::D, (cuuint32_t)p.page, 1, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, box,
                   estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// Blocks of a decode cluster: the largest power of two that leaves no more than 1.3 waves of
// blocks (two to an SM), 0 when the statistics of the longest sequence do not fit. More splits a
// long sequence finer but adds blocks that cost 8 us each and run in a second wave. The host knows
// how many sequences there are, not how long each is, and the best size depends on both; the rule
// favours ragged batches, whose short sequences leave the second wave room. In us, the chosen size
// first, groups = sequences x 8 heads:
//   24 ragged to 16384 (192 groups), tau = 1 (and 0): 2 blocks 39 (60), 1: 59 (106), 4: 45 (43)
//   uniform, 8192 keys, tau = 0:  40 groups: 8 blocks 27, 4: 24, 16: 33;  80: 4 blocks 44, 2: 39,
//     8: 43;  128: 2 blocks 47, 4: 57;  160: 2 blocks 78, 1: 67, 4: 70;  192: 2 blocks 80, 1: 71;
//     256: 1 block 83;  320: 1 block 141 (24 blocks run a second wave alone), 2: 125, 4: 121;
//     384: 1 block 147, 2: 132;  512: 1 block 161
//   and tau = 1:  40: 8 blocks 29, 4: 20;  80: 4 blocks 42, 2: 31;  160: 2 blocks 65, 1: 52;  192:
//     2 blocks 68, 1: 57;  320: 1 block 109, 2: 105
// So a uniform batch just above a whole wave pays up to 1.2 times (tau = 1: 1.4) for what a ragged
// one gains. Clusters of 16 blocks do not pack: the chip holds 14, not 18, so they are for fewer groups than
// that (16 groups of 16384 keys: 8 blocks 41 us, 16: 59 us).
inline int decode_cluster(const pdec::Params& p, long long groups, bool rule, size_t* smem) {
  int best = 0;
  for (int C = 1; C <= pdec::MAXC; C *= 2) {
    const size_t need = pdec::smem_bytes(p.G, p.max_tiles, C, p.per_head, rule);
    if (need > pdec::MAX_SMEM) continue;
    const long long slots = (long long)sm_count() * (need <= 113 * 1024 ? 2 : 1);
    const long long room = C == 16 ? 10 * slots / 13 : 13 * slots / 10;
    if (best > 0 && (groups * C > room || C / 2 >= p.max_tiles)) break;
    best = C;
    *smem = need;
  }
  return best;
}

// What a decode kernel may use, said once per device and context: three calls of the runtime for
// each step would be a tenth of its host time. Remembered is the context that it was said in: after
// cudaDeviceReset it has to be said again, or the launch is refused.
inline bool allow_decode(pdec::Kernel kernel, bool wide, bool rule) {
  constexpr int kDevices = 64;
  static std::atomic<unsigned long long> said[2][2][kDevices];
  int dev = 0;
  unsigned long long ctx = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || !current_context_id(&ctx)) return false;
  std::atomic<unsigned long long>* mine = dev < kDevices ? &said[wide][rule][dev] : nullptr;
  if (mine && ctx != 0 && mine->load(std::memory_order_relaxed) == ctx) return true;
  // the carve-out: without it an SM takes one block, although the shared memory of two fits
  const bool ok =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)pdec::MAX_SMEM) == cudaSuccess &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) ==
          cudaSuccess &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                           cudaSharedmemCarveoutMaxShared) == cudaSuccess;
  if (ok && mine && ctx != 0) mine->store(ctx, std::memory_order_relaxed);
  return ok;
}

// An input or output of append: [total][heads][128] bf16 by its strides.
inline bool rows_ok(const void* ptr, int64_t token_stride, int64_t head_stride) {
  return ptr && aligned16(ptr) && !(token_stride & 7) && !(head_stride & 7);
}

}  // namespace host
}  // namespace mala

extern "C" {

mala_status mala_cache_append(const mala_paged_cache* cache, const void* k, int64_t k_token_stride,
                              int64_t k_head_stride, const void* v, int64_t v_token_stride,
                              int64_t v_head_stride, const void* q, int64_t q_token_stride,
                              int64_t q_head_stride, void* q_out, int64_t q_out_token_stride,
                              int64_t q_out_head_stride, const int32_t* cu_seqlens,
                              const int32_t* seq_lens, int batch, int total, int max_new, int Hq,
                              const float* inv_freq, int rot_dim, int interleaved, void* stream) {
  mala::paged::AppendParams p = {};
  const mala_status st = make_pool(cache, &p.pool);
  if (st != MALA_OK) return st;
  const int Hkv = cache->Hkv;
  if (batch < 1 || total < 0 || max_new < 0 || (interleaved != 0 && interleaved != 1))
    return MALA_ERR_INVALID_ARG;
  if (batch > 65535 || (q && (Hq < 1 || Hq % Hkv != 0))) return MALA_ERR_INVALID_ARG;
  if (rot_dim < 0 || rot_dim > mala::paged::D || rot_dim % 16 != 0) return MALA_ERR_UNSUPPORTED;
  if (!cu_seqlens && total != batch) return MALA_ERR_INVALID_ARG;
  if (!seq_lens || (rot_dim > 0 && !inv_freq)) return MALA_ERR_INVALID_ARG;
  const void* words[] = {cu_seqlens, seq_lens, inv_freq};
  for (const void* w : words)
    if (reinterpret_cast<uintptr_t>(w) & 3u) return MALA_ERR_INVALID_ARG;
  if (total == 0 || max_new == 0) return MALA_OK;
  if (!rows_ok(k, k_token_stride, k_head_stride) || !rows_ok(v, v_token_stride, v_head_stride))
    return MALA_ERR_INVALID_ARG;
  if (q && (!rows_ok(q, q_token_stride, q_head_stride) ||
            !rows_ok(q_out, q_out_token_stride, q_out_head_stride)))
    return MALA_ERR_INVALID_ARG;
  p.k = reinterpret_cast<const __nv_bfloat16*>(k);
  p.v = reinterpret_cast<const __nv_bfloat16*>(v);
  p.q = reinterpret_cast<const __nv_bfloat16*>(q);
  p.q_out = reinterpret_cast<__nv_bfloat16*>(q_out);
  p.k_tok = k_token_stride;
  p.k_head = k_head_stride;
  p.v_tok = v_token_stride;
  p.v_head = v_head_stride;
  p.q_tok = q_token_stride;
  p.q_head = q_head_stride;
  p.qo_tok = q_out_token_stride;
  p.qo_head = q_out_head_stride;
  p.cu = cu_seqlens;
  p.seq_lens = seq_lens;
  p.inv_freq = inv_freq;
  p.rot = rot_dim;
  p.G = q ? Hq / Hkv : 0;
  p.total = total;
  p.max_new = max_new < total ? max_new : total;
  const int page = cache->page_size;
  // n consecutive positions lie in at most (n + page - 2) / page + 1 pages
  const long long pages = ((long long)p.max_new + page - 2) / page + 1;
  const int rows = page < p.max_new ? page : p.max_new;  // new ones of a page
  const int half = p.rot / 2;
  cudaStream_t s = as_stream(stream);
  // A block's heads: all when there are pages enough to fill the chip four times, so that they
  // share the angles; of decode steps as many as make 32 units of eight threads.
  int groups = 1;
  if (rows <= 2) {
    const int each = 32 / (2 + p.G) > 1 ? 32 / (2 + p.G) : 1;
    groups = (Hkv + each - 1) / each;
  } else {
    const long long blocks = (long long)batch * pages, want = 4ll * sm_count();
    if (blocks < want) groups = (int)((want + blocks - 1) / blocks);
  }
  groups = groups < Hkv ? groups : Hkv;
  p.heads = (Hkv + groups - 1) / groups;
  const dim3 grid((unsigned)pages, batch, (Hkv + p.heads - 1) / p.heads);
  const size_t table = half > 0 && rows > 2 ? (size_t)rows * 32 * sizeof(float4) : 0;
  const mala::paged::AppendKernel kernel = mala::paged::append_kernel_of(rows, interleaved != 0);
  if (table > 48 * 1024)
    MALA_CUDA_TRY(
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)table));
  kernel<<<grid, mala::paged::APPEND_NT, table, s>>>(p);
  return launch_status();
}

mala_status mala_decode_paged(const mala_paged_cache* cache, const void* q, void* o,
                              const int32_t* seq_lens, int batch, int Hq, int max_seqlen,
                              float tau, float scale, int per_head, int32_t* kept_tiles,
                              uint32_t* keep_bits, void* stream) {
  mala::pdec::Params p = {};
  const mala_status st = make_pool(cache, &p.pool);
  if (st != MALA_OK) return st;
  const int Hkv = cache->Hkv;
  if (batch < 1 || batch > 65535 || Hq < 1 || Hq % Hkv != 0) return MALA_ERR_INVALID_ARG;
  if (per_head != 0 && per_head != 1) return MALA_ERR_INVALID_ARG;
  if (!tau_ok(tau)) return MALA_ERR_INVALID_ARG;
  if (Hq / Hkv > mala::pdec::GMAX) return MALA_ERR_UNSUPPORTED;
  if (!q || !o || !seq_lens || !aligned16(q) || !aligned16(o)) return MALA_ERR_INVALID_ARG;
  const void* words[] = {seq_lens, kept_tiles, keep_bits};
  for (const void* w : words)
    if (reinterpret_cast<uintptr_t>(w) & 3u) return MALA_ERR_INVALID_ARG;
  const int held = cache->max_pages * cache->page_size;
  if (max_seqlen <= 0) max_seqlen = held;
  p.nw = (int)(((long long)max_seqlen + 4095) / 4096);  // trace rows: the caller's max_seqlen
  p.max_len = max_seqlen < held ? max_seqlen : held;
  p.max_tiles = (p.max_len + 127) / 128;
  p.q = reinterpret_cast<const __nv_bfloat16*>(q);
  p.o = reinterpret_cast<__nv_bfloat16*>(o);
  p.seq_lens = seq_lens;
  p.G = Hq / Hkv;
  p.GP = (p.G + 1) & ~1;
  p.Hkv = Hkv;
  p.scale_log2 = resolve_scale(scale, mala::paged::D) * mala::kLog2e;
  p.log2_tau = tau > 0.f ? log2f(tau) : 0.f;
  p.per_head = per_head;
  p.kept_tiles = kept_tiles;
  p.keep_bits = keep_bits;
  CUtensorMap mk, mv;
  if (!make_page_map(&mk, p.pool.k, p.pool, p.pool.k_page, p.pool.k_head, p.pool.k_tok) ||
      !make_page_map(&mv, p.pool.v, p.pool, p.pool.v_page, p.pool.v_head, p.pool.v_tok))
    return MALA_ERR_CUDA;
  // a single tile is always kept: exact attention is the rule's answer
  const bool rule = tau > 0.f && p.max_tiles > 1;
  const mala::pdec::Kernel kernel = mala::pdec::decode_kernel_of(p.G, rule);
  if (!allow_decode(kernel, p.G > 4, rule)) return MALA_ERR_CUDA;
  size_t smem;
  p.C = decode_cluster(p, (long long)batch * Hkv, rule, &smem);
  if (p.C < 1) return MALA_ERR_TOO_LARGE;
  while (1 << p.C_log2 < p.C) ++p.C_log2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.C, Hkv, batch);
  cfg.blockDim = dim3(mala::pdec::NT, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = as_stream(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  MALA_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, mk, mv, p));
  return launch_status();
}

mala_status mala_cache_gather(const mala_paged_cache* cache, void* K, void* V,
                              const int32_t* cu_seqlens_k, int batch, int max_seqlen, int total,
                              void* stream) {
  mala::paged::GatherParams p = {};
  const mala_status st = make_pool(cache, &p.pool);
  if (st != MALA_OK) return st;
  if (batch < 1 || batch > 65535 || total < 0 || max_seqlen < 0) return MALA_ERR_INVALID_ARG;
  if (!cu_seqlens_k || (reinterpret_cast<uintptr_t>(cu_seqlens_k) & 3u))
    return MALA_ERR_INVALID_ARG;
  if (total == 0 || max_seqlen == 0) return MALA_OK;
  if (!K || !V || !aligned16(K) || !aligned16(V)) return MALA_ERR_INVALID_ARG;
  p.k = reinterpret_cast<__nv_bfloat16*>(K);
  p.v = reinterpret_cast<__nv_bfloat16*>(V);
  p.cu = cu_seqlens_k;
  p.total = total;
  p.max_seqlen = max_seqlen < total ? max_seqlen : total;
  const int page = cache->page_size;
  const dim3 grid((p.max_seqlen - 1) / page + 1, batch);
  mala::paged::gather_kernel<<<grid, mala::paged::GATHER_NT, 0, as_stream(stream)>>>(p);
  return launch_status();
}

}  // extern "C"
