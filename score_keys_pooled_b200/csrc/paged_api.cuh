// C ABI of the rotation, the paged-cache append and the paged attention:
// argument checks, workspace layout and launches.  Included by s2o_api.cu,
// whose helpers (alignment, tensor-map encoder, launch count) it uses.
#pragma once

namespace {

constexpr double kPerTurn = 0.15915494309189533576888376337251;  // 1 / (2 pi)

s2o_status rotary_table(const s2o_rotary_config* r, bool inverse, RotaryTable* t) {
  std::memset(t, 0, sizeof(*t));
  t->sign = inverse ? -1.f : 1.f;
  if (!r) return S2O_OK;  // no rotation
  if (r->rot_dim < 0 || r->naxes < 1 || r->naxes > 3) return S2O_ERR_INVALID_ARG;
  if (r->rot_dim % 16 || r->rot_dim > kD) return S2O_ERR_UNSUPPORTED_SHAPE;
  t->rot = r->rot_dim;
  t->adjacent = r->interleaved != 0;
  t->naxes = r->naxes;
  for (int i = 0; i < r->rot_dim / 2; ++i) {
    if (!std::isfinite(r->inv_freq[i]) || r->axis[i] >= r->naxes) return S2O_ERR_INVALID_ARG;
    t->turns[i] = r->inv_freq[i] * kPerTurn;
    t->axis[i] = r->axis[i];
  }
  return S2O_OK;
}

// A view of B x N x H rows.  Rows stay 16-byte aligned; a stride that no row is
// reached by says nothing.
bool take_view(const s2o_view* v, int64_t B, int64_t N, int64_t H, RowView* out) {
  if (!v->ptr || !aligned16(v->ptr)) return false;
  out->p = static_cast<uint16_t*>(v->ptr);
  out->sb = B > 1 ? v->stride_b : 0;
  out->st = N > 1 ? v->stride_t : 0;
  out->sh = H > 1 ? v->stride_h : 0;
  return out->sb % 8 == 0 && out->st % 8 == 0 && out->sh % 8 == 0;
}

// an output where the input it is made from has other rows: in place means in
// every row's own place
bool rows_clash(const RowView& out, const RowView& in, int64_t B, int64_t N, int64_t H) {
  return !rows_same(out, in, B, N, H) && rows_meet(out, H, in, H, B, N);
}
// [a, a + an) and [b, b + bn) bytes share one
bool ranges_meet(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + bn && y < x + an;
}

s2o_status check_cache(const s2o_cache_config* c) {
  if (!c) return S2O_ERR_INVALID_ARG;
  if (c->Hq <= 0 || c->Hkv <= 0 || c->d <= 0 || c->page_size <= 0 || c->num_pages <= 0 || c->nseq <= 0 ||
      c->max_pages <= 0 || c->Tq < 0 || c->max_q <= 0 || c->prefix_len < 0 || c->Hq % c->Hkv)
    return S2O_ERR_INVALID_ARG;
  if (c->dtype != S2O_TYPE_BF16 && c->dtype != S2O_TYPE_FP16) return S2O_ERR_INVALID_ARG;
  if (c->d != kD) return S2O_ERR_UNSUPPORTED_SHAPE;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
    return S2O_ERR_UNSUPPORTED_SHAPE;
  // row numbers of the caches are 32-bit coordinates, key numbers 32-bit
  if ((int64_t)c->num_pages * c->Hkv * c->page_size >= (int64_t)INT32_MAX ||
      (int64_t)c->max_pages * c->page_size + c->prefix_len >= (int64_t)INT32_MAX - 512)
    return S2O_ERR_UNSUPPORTED_SHAPE;
  if (c->Hq / c->Hkv > 64 || (int64_t)c->Tq * c->Hq >= (int64_t)INT32_MAX) return S2O_ERR_UNSUPPORTED_SHAPE;
  return S2O_OK;
}

int log2_of(int x) {
  int l = 0;
  while ((1 << l) < x) ++l;
  return l;
}

int sm_count() {
  int dev = 0, n = 148;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n;
}

// The paged attention's kernels for a call: a rule on sizes the host knows, so
// the workspace size and the launches agree.
//
// Rows of a sequence's new tokens (max_q G) up to 32 go to the decode kernel,
// which reads the cache at 16 or 32 rows a key; more fill a tcgen05 tile well
// enough (33 rows of 128 still keep up with the memory: 64 KB of keys in 1.3
// us).  The prefix is then taken the cheapest of these ways:
//   walk    each own item begins with the prefix: one list of parts, but every
//           item reads it (from L2 where it fits)
//   items   prefix items in the same kernel: read once per row tile
//   tiles   (decode) prefix items in the tile kernel beside it
// By what each costs beside the own keys, in microseconds:
//   units   an SM's 128 keys in the tile kernel kTileNs, kHalfTileNs with 128
//           rows (1.75 us where every item reads them for itself: 64 KB a unit
//           on all SMs are 5.5 TB/s); 64 in the decode kernel 1.2, with four
//           streams 1.7 (the join of a token's many parts among it)
//   walk    the row tiles of ragged sequences are at most one each and one more
//           for every tpt tokens, and at most the tiles of max_q each; in the
//           tile kernel 0.2 for each part that few long items are cut into
//   items   the second list of parts: 2 and 1.5 a thousand rows, in the tile
//           kernel 2 and 0.5
//   tiles   as items, and 8.5 for a second kernel beside the first
// 561 shapes with each way forced (1 to 256 sequences of 1 to 1023 new tokens,
// prefixes of 10 to 131072, groups of 1 to 8): the way taken is within 3 % of the
// best on 505, 0.9 % behind it on average, 20 % at most (one chunk of 44 tokens
// with 22000 own keys behind 89: 41.0 us where items take 34.0).  Walk, items,
// tiles at 32 heads on 8: 16 sequences of one token behind 1000 26.0, 23.4, 24.6 us,
// behind 4000 43, 27.5, 27.8, behind 20000 134, 54, 39; 16 of 4 tokens behind 1000
// 28.0, 27.1, 25.1; 32 chunks of 64 behind 8000 271, 303, behind 32768 1091, 1130;
// one of 512 and 63 single tokens behind 8192 539, 136.
struct PagedPlan {
  bool chunks;   // the tile kernel takes the own keys, otherwise the decode kernel
  bool tiles;    // decode: the tile kernel takes the prefix beside it
  bool direct;   // whole items are the result
  int R;         // row tiles of 16 of the decode kernel
  PagedCut tile, decode;
};
PagedPlan paged_plan(const s2o_cache_config* c, int sms) {
  PagedPlan p{};
  const int G = c->Hq / c->Hkv;
  const int max_q = std::min(c->max_q, std::max(c->Tq, 1));
  const int64_t seq_rows = (int64_t)max_q * G;
  p.chunks = seq_rows > 32;
  p.R = seq_rows <= 16 ? 1 : 2;
  p.tile.tpt = 2 * (kLq / G);
  p.tile.kt_log2 = 7;
  p.decode.tpt = std::max(1, 16 * p.R / G);
  p.decode.kt_log2 = 6;
  // what a piece costs beside its keys (see `fixed`): in the tile kernel 4 us,
  // the row sums' way out of tensor memory (33 sequences of 40 rows, 700 keys,
  // behind 5001: 36.9, 34.4, 32.8, 34.0 us with 0, 1, 2, 3 units)
  p.tile.fixed = 2;
  p.decode.fixed = 1;
  PagedCut& own = p.chunks ? p.tile : p.decode;
  own.own_items = 1;
  // microseconds
  const double prefix = c->prefix_len, tokens = c->Tq, seqs = std::min(c->nseq, std::max(c->Tq, 1));
  const double units = c->Hkv * std::ceil(prefix / (1 << own.kt_log2)) / sms;
  const double tile = (2 * tokens <= p.tile.tpt ? kHalfTileNs : kTileNs) * 1e-3, krows = 1e-3 * tokens * c->Hq;
  const double own_tiles = std::min(seqs + std::floor((tokens - seqs) / own.tpt), seqs * std::ceil((double)max_q / own.tpt));
  const double tok_tiles = std::ceil(tokens / own.tpt);
  double walk, items, tiles = INFINITY;
  if (p.chunks) {
    const double parts = std::min(sms / (own_tiles * c->Hkv), std::ceil(prefix / 128) + own.fixed);
    walk = units * own_tiles * (2 * max_q <= own.tpt ? 1.75 : kTileNs * 1e-3) + 0.2 * std::max(0., parts - 1);
    items = units * tok_tiles * tile + 2 + 0.5 * krows;
  } else {
    const double unit = p.R == 1 ? 1.2 : 1.7, join = 2 + 1.5 * krows;
    walk = units * own_tiles * unit;
    items = units * tok_tiles * unit + join;
    tiles = c->Hkv * std::ceil(prefix / 128) / sms * std::ceil(tokens / p.tile.tpt) * tile + join + 8.5;
  }
  p.direct = c->prefix_len == 0 || (walk <= items && walk <= tiles);
  p.tiles = !p.direct && tiles < items;
  own.walk_prefix = p.direct && c->prefix_len > 0;
  own.prefix_items = !p.direct && !p.tiles;
  p.tile.prefix_items |= p.tiles;
  return p;
}

struct PagedWs {
  PagedHead* head;  // of the tile kernel, of the decode kernel
  int4* meta;
  SplitItem* split;
  PagedPart tile, decode;
  size_t bytes;
};
// workers of the kernel that takes the own keys
int own_workers(const PagedPlan& p, int sms) { return p.chunks ? sms : sms * (kPgWarps / p.R); }

PagedWs paged_layout(const s2o_cache_config* c, const PagedPlan& p, int n, void* base) {
  PagedWs w{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    uint8_t* q = static_cast<uint8_t*>(base) + off;
    off += round256(bytes);
    return static_cast<void*>(q);
  };
  const size_t rows = (size_t)c->Tq * c->Hq;
  w.head = static_cast<PagedHead*>(take(2 * sizeof(PagedHead)));
  if (p.direct && p.chunks) w.split = static_cast<SplitItem*>(take((size_t)n * sizeof(SplitItem)));
  else w.meta = static_cast<int4*>(take((size_t)c->Tq * c->Hkv * sizeof(int4)));
  if (!p.direct) {
    for (int k = 0; k < 2; ++k) {
      w.decode.dense[k] = static_cast<float*>(take(rows * kD * sizeof(float)));
      w.decode.dense_ml[k] = static_cast<float2*>(take(rows * sizeof(float2)));
    }
  }
  w.tile = w.decode;
  auto slots = [&](PagedPart& part, int workers, int r) {
    part.rows = r;
    part.slots = static_cast<float*>(take((size_t)2 * workers * r * kD * sizeof(float)));
    part.slots_ml = static_cast<float2*>(take((size_t)2 * workers * r * sizeof(float2)));
  };
  if (p.chunks || p.tiles) slots(w.tile, n, 2 * kLq);
  if (!p.chunks) slots(w.decode, own_workers(p, n), 16 * p.R);
  w.bytes = off;
  return w;
}

// [Tq, Hq, 128] queries as boxes of 64 columns x G heads x `toks` tokens
bool encode_query_map(CUtensorMap* map, const void* base, int Tq, int Hq, int G, int toks, bool fp16) {
  EncodeTiledFn enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)kD, (cuuint64_t)Hq, (cuuint64_t)Tq};
  const cuuint64_t strides[2] = {(cuuint64_t)kD * 2, (cuuint64_t)Hq * kD * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)toks};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
             const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// launch that may start before the kernel in front of it is done
// (an error is taken off the runtime's record: it is this call's to report)
template <class... P, class... A>
cudaError_t launch_early(void (*f)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t s, bool early,
                         const A&... args) {
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &at;
  cfg.numAttrs = early ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, f, args...);
  if (e != cudaSuccess) cudaGetLastError();
  return e;
}

template <class F>
cudaError_t allow_smem(F f, size_t bytes) {
  // the attribute belongs to the function on the current device; setting it
  // again costs less than a microsecond
  const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e != cudaSuccess) cudaGetLastError();
  return e;
}

template <bool FP16>
cudaError_t launch_tile(const PagedArgs& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, int n,
                        cudaStream_t s) {
  const cudaError_t e = allow_smem(k_paged_tile<FP16>, kPtSmem);
  if (e != cudaSuccess) return e;
  return launch_early(k_paged_tile<FP16>, n, kAttn2Threads, kPtSmem, s, false, a, q, k, v);
}
template <bool FP16, int R>
cudaError_t launch_decode(const PagedArgs& a, const CUtensorMap& k, const CUtensorMap& v, int n, cudaStream_t s,
                          bool early) {
  const cudaError_t e = allow_smem(k_paged_decode<FP16, R>, PgDecode<R>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_early(k_paged_decode<FP16, R>, n, 32 * kPgWarps, PgDecode<R>::kSmem, s, early, a, k, v);
}
template <bool FP16>
cudaError_t launch_decode_r(int R, const PagedArgs& a, const CUtensorMap& k, const CUtensorMap& v, int n,
                            cudaStream_t s, bool early) {
  return R == 1 ? launch_decode<FP16, 1>(a, k, v, n, s, early) : launch_decode<FP16, 2>(a, k, v, n, s, early);
}

}  // namespace

extern "C" {

s2o_status s2o_rotary(const s2o_rotary_config* rotary, int32_t dtype, int32_t B, int32_t N, int32_t Hq, int32_t Hkv,
                      const s2o_view* q, const s2o_view* k, const int32_t* positions, const s2o_view* q_out,
                      const s2o_view* k_out, int32_t inverse, s2o_stream_t stream) {
  t_launches = 0;
  if (!rotary || B < 0 || N < 0 || Hq < 0 || Hkv < 0 || (dtype != S2O_TYPE_BF16 && dtype != S2O_TYPE_FP16))
    return S2O_ERR_INVALID_ARG;
  RotaryArgs a;
  s2o_status st = rotary_table(rotary, inverse != 0, &a.r);
  if (st != S2O_OK) return st;
  if (B == 0 || N == 0 || Hq + (int64_t)Hkv == 0) return S2O_OK;
  if ((int64_t)Hq + Hkv > 4096) return S2O_ERR_UNSUPPORTED_SHAPE;
  if (!positions || (Hq && (!q || !q_out)) || (Hkv && (!k || !k_out))) return S2O_ERR_INVALID_ARG;
  std::memset(&a.q, 0, 4 * sizeof(RowView));
  if (Hq && (!take_view(q, B, N, Hq, &a.q) || !take_view(q_out, B, N, Hq, &a.qo))) return S2O_ERR_INVALID_ARG;
  if (Hkv && (!take_view(k, B, N, Hkv, &a.k) || !take_view(k_out, B, N, Hkv, &a.ko))) return S2O_ERR_INVALID_ARG;
  // rows are turned in any order: none may be written twice, or before another is made from it
  if ((Hq && (rows_meet(a.qo, B, N, Hq) || rows_clash(a.qo, a.q, B, N, Hq))) ||
      (Hkv && (rows_meet(a.ko, B, N, Hkv) || rows_clash(a.ko, a.k, B, N, Hkv))) ||
      (Hq && Hkv && (rows_meet(a.qo, Hq, a.ko, Hkv, B, N) || rows_meet(a.qo, Hq, a.k, Hkv, B, N) ||
                     rows_meet(a.q, Hq, a.ko, Hkv, B, N))))
    return S2O_ERR_INVALID_ARG;
  a.pos = positions;
  a.B = B; a.N = N; a.Hq = Hq; a.Hkv = Hkv;
  const int64_t total = (int64_t)B * N;
  a.tb = kRotMaxTokens;
  while (a.tb > 1 && total < (int64_t)a.tb * 148 * 4) a.tb >>= 1;
  const int64_t blocks = (total + a.tb - 1) / a.tb;
  if (blocks > INT32_MAX) return S2O_ERR_UNSUPPORTED_SHAPE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == S2O_TYPE_FP16) k_rotary<true><<<(unsigned)blocks, kRotThreads, 0, s>>>(a);
  else k_rotary<false><<<(unsigned)blocks, kRotThreads, 0, s>>>(a);
  ++t_launches;
  return launch_status();
}

s2o_status s2o_cache_append(const s2o_cache_config* cfg, const s2o_rotary_config* rotary, const s2o_view* q,
                            const s2o_view* k, const s2o_view* v, const int32_t* positions, const int32_t* page_table,
                            const int32_t* q_start, const int32_t* kv_len, uint16_t* k_cache, uint16_t* v_cache,
                            const s2o_view* q_out, s2o_stream_t stream) {
  t_launches = 0;
  s2o_status st = check_cache(cfg);
  if (st != S2O_OK) return st;
  AppendArgs a;
  st = rotary_table(rotary, false, &a.r);
  if (st != S2O_OK) return st;
  if (cfg->Tq == 0) return S2O_OK;  // nothing to write; the tensors may have no memory
  if (!k || !v || !page_table || !q_start || !kv_len || !k_cache || !v_cache || !q != !q_out)
    return S2O_ERR_INVALID_ARG;
  if (!aligned16(k_cache) || !aligned16(v_cache)) return S2O_ERR_INVALID_ARG;
  std::memset(&a.q, 0, 4 * sizeof(RowView));
  const int T = cfg->Tq, Hq = cfg->Hq, Hkv = cfg->Hkv;
  if (!take_view(k, 1, T, Hkv, &a.k) || !take_view(v, 1, T, Hkv, &a.v)) return S2O_ERR_INVALID_ARG;
  if (q && (!take_view(q, 1, T, Hq, &a.q) || !take_view(q_out, 1, T, Hq, &a.qo) || rows_meet(a.qo, 1, T, Hq) ||
            rows_clash(a.qo, a.q, 1, T, Hq) || rows_meet(a.qo, Hq, a.k, Hkv, 1, T) || rows_meet(a.qo, Hq, a.v, Hkv, 1, T)))
    return S2O_ERR_INVALID_ARG;
  const size_t cache = (size_t)cfg->num_pages * Hkv * cfg->page_size * kD * sizeof(uint16_t);
  if (ranges_meet(k_cache, cache, v_cache, cache)) return S2O_ERR_INVALID_ARG;
  if ((int64_t)cfg->Hq + 2 * (int64_t)cfg->Hkv > 4096) return S2O_ERR_UNSUPPORTED_SHAPE;
  a.pos = positions;
  a.table = page_table; a.q_start = q_start; a.kv_len = kv_len;
  a.kc = k_cache; a.vc = v_cache;
  a.Hq = cfg->Hq; a.Hkv = cfg->Hkv; a.page_log2 = log2_of(cfg->page_size); a.num_pages = cfg->num_pages;
  a.nseq = cfg->nseq; a.max_pages = cfg->max_pages; a.Tq = cfg->Tq; a.max_q = cfg->max_q; a.prefix = cfg->prefix_len;
  a.tb = kRotMaxTokens;
  while (a.tb > 1 && cfg->Tq < a.tb * 148 * 4) a.tb >>= 1;
  const unsigned blocks = ((unsigned)cfg->Tq + a.tb - 1) / a.tb;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (cfg->dtype == S2O_TYPE_FP16) k_cache_append<true><<<blocks, kRotThreads, 0, s>>>(a);
  else k_cache_append<false><<<blocks, kRotThreads, 0, s>>>(a);
  ++t_launches;
  return launch_status();
}

s2o_status s2o_attention_paged_workspace_size(const s2o_cache_config* cfg, size_t* bytes) {
  s2o_status st = check_cache(cfg);
  if (st != S2O_OK) return st;
  if (!bytes) return S2O_ERR_INVALID_ARG;
  const int n = sm_count();
  *bytes = paged_layout(cfg, paged_plan(cfg, n), n, nullptr).bytes;
  return S2O_OK;
}

s2o_status s2o_attention_paged(const s2o_cache_config* cfg, const uint16_t* Q, const uint16_t* k_cache,
                               const uint16_t* v_cache, const int32_t* prefix_pages, const int32_t* page_table,
                               const int32_t* q_start, const int32_t* kv_len, void* O, int32_t out_dtype, float* lse,
                               void* workspace, size_t workspace_bytes, s2o_stream_t stream) {
  t_launches = 0;
  s2o_status st = check_cache(cfg);
  if (st != S2O_OK) return st;
  if (cfg->Tq == 0) return S2O_OK;  // no rows; the tensors may have no memory
  if (!Q || !k_cache || !v_cache || !page_table || !q_start || !kv_len || !O || !workspace ||
      (cfg->prefix_len > 0 && !prefix_pages))
    return S2O_ERR_INVALID_ARG;
  if (out_dtype != S2O_OUT_SAME && out_dtype != S2O_OUT_F32) return S2O_ERR_INVALID_ARG;
  if (!aligned16(Q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(O) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return S2O_ERR_INVALID_ARG;
  const size_t rows = (size_t)cfg->Tq * cfg->Hq, row = kD * sizeof(uint16_t);
  if (ranges_meet(O, rows * row * (out_dtype == S2O_OUT_F32 ? 2 : 1), Q, rows * row)) return S2O_ERR_INVALID_ARG;
  const int n = sm_count();
  const PagedPlan p = paged_plan(cfg, n);
  const PagedWs w = paged_layout(cfg, p, n, workspace);
  if (workspace_bytes < w.bytes) return S2O_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  PagedArgs a{};
  PagedGeom& g = a.g;
  g.table = page_table; g.prefix_pages = prefix_pages; g.q_start = q_start; g.kv_len = kv_len;
  g.Hq = cfg->Hq; g.Hkv = cfg->Hkv; g.G = cfg->Hq / cfg->Hkv; g.nseq = cfg->nseq; g.max_pages = cfg->max_pages;
  g.num_pages = cfg->num_pages; g.page_log2 = log2_of(cfg->page_size); g.Tq = cfg->Tq; g.max_q = cfg->max_q;
  g.prefix = cfg->prefix_len;
  a.Q = Q; a.O = O; a.lse = lse; a.meta = w.meta; a.split = w.split;
  a.out_f32 = out_dtype == S2O_OUT_F32;
  a.direct = p.direct;
  a.beside = p.tiles;
  a.own_ns = p.R == 1 ? 520.f : 1100.f;
  CUtensorMap tmQ, tmK, tmV;
  const uint64_t cache_rows = (uint64_t)cfg->num_pages * cfg->Hkv * cfg->page_size;
  const uint32_t box = (uint32_t)std::min(cfg->page_size, 64);
  const bool fp16 = cfg->dtype == S2O_TYPE_FP16;
  if (p.chunks || p.tiles) {
    if (!encode_rows_map(&tmK, k_cache, cache_rows, box) || !encode_rows_map(&tmV, v_cache, cache_rows, box)) return S2O_ERR_CUDA;
    if (!encode_query_map(&tmQ, Q, cfg->Tq, cfg->Hq, g.G, kLq / g.G, fp16)) return S2O_ERR_CUDA;
    a.c = p.tile;
    a.other = p.decode;
    a.part = w.tile;
    a.head = w.head;
    if ((fp16 ? launch_tile<true>(a, tmQ, tmK, tmV, n, s) : launch_tile<false>(a, tmQ, tmK, tmV, n, s)) != cudaSuccess)
      return S2O_ERR_CUDA;
    ++t_launches;
  }
  if (!p.chunks) {
    if (!encode_rows_map(&tmK, k_cache, cache_rows, kPgSub) || !encode_rows_map(&tmV, v_cache, cache_rows, kPgSub))
      return S2O_ERR_CUDA;
    a.c = p.decode;
    a.other = p.tile;
    a.part = w.decode;
    a.head = w.head + 1;
    // beside the tile kernel: neither reads what the other writes
    if ((fp16 ? launch_decode_r<true>(p.R, a, tmK, tmV, n, s, p.tiles)
              : launch_decode_r<false>(p.R, a, tmK, tmV, n, s, p.tiles)) != cudaSuccess)
      return S2O_ERR_CUDA;
    ++t_launches;
  }
  JoinArgs j{};
  j.g = g;
  const JoinSide tile = {w.tile, p.tile, w.head, n}, decode = {w.decode, p.decode, w.head + 1, own_workers(p, n)};
  j.own = p.chunks ? tile : decode;
  j.prefix = p.tiles ? tile : j.own;
  j.meta = w.meta; j.split = w.split; j.O = O; j.lse = lse; j.out_f32 = a.out_f32;
  j.direct = p.direct;
  cudaError_t e;
  if (w.split) {
    const dim3 grid(n, 32);
    e = launch_early(fp16 ? k_paged_join_split<true> : k_paged_join_split<false>, grid, 32 * kJoinWarps, 0, s, true, j);
  } else {
    const int64_t nrows = (int64_t)cfg->Tq * cfg->Hq;
    const bool many = nrows > (int64_t)n * 8;  // more than one wave of a block each
    const unsigned blocks = (unsigned)(many ? (nrows + kJoinWarps - 1) / kJoinWarps : nrows);
    e = launch_early(fp16 ? (many ? k_paged_join<true, true> : k_paged_join<true, false>)
                          : (many ? k_paged_join<false, true> : k_paged_join<false, false>), blocks, 32 * kJoinWarps, 0, s, true, j);
  }
  if (e != cudaSuccess) return S2O_ERR_CUDA;
  ++t_launches;
  return S2O_OK;
}

}  // extern "C"
