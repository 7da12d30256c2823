// Attention over a paged cache, up to 32 query rows a sequence and KV head: one
// token or a few drafted ones of every sequence against their own keys, and
// against a shared prefix where the tile kernel (paged_tile.cuh) does not take
// it.  The join of partial results, of either kernel, is at the end.
//
//   o_i = sum_j exp(s_ij) v_j / sum_j exp(s_ij),  s_ij = q_i . k_j / sqrt(d),
//   j over the prefix and the own keys up to the row's own
//
// Bound by the cache: a key and its value are 512 bytes for 4 d flops a row,
// 16 flops a byte at 16 rows, far below what the GPU can do, so the kernel is
// built to keep reads in flight and to have nothing wait for anything else:
//
//   * a CTA (one per SM, 8 warps) is 8 / R independent streams of R warps.  A
//     stream is a worker with a share of its own (paged_sched.cuh): it walks
//     its keys 16 at a time through its own ring of 8 KB stages (192 KB of
//     stages per SM), and its first warp issues the TMA boxes itself, each
//     into the stage that the stream has just read.  A stage costs a stream 0.7
//     to 0.9 us of latency (two chains of products with the softmax between)
//     and a piece 2.2 us (sequence numbers, first loads, results), while the
//     other streams' reads go on: 16 sequences of up to 32K keys, 1.07 GB, take
//     187 us, 5.8 TB/s, 88 % of the measured copy rate; even shares on SMs that
//     are not equally near the memory (warps end between 119 and 174 us) are
//     what is left.  One ring for the whole CTA, its 64-key stages cut into
//     slices over four or eight warps and joined in shared memory at the end of
//     each piece, spent 8 to 13 us at every piece boundary: 58 and 79 us on 64
//     sequences of 512 keys where this takes 45.
//   * a warp holds 16 query rows (an mma's M), their running reference and
//     sum, and a 16 x 128 fp32 accumulator in registers; with R = 2 two warps
//     of a stream hold 32 rows against the same stages.
//   * products: mma.sync m16n8k16 (bf16 or fp16 in, fp32 out).  With at most
//     32 rows a KV head the 128-row tcgen05 tile would be mostly empty and
//     its round trip through tensor memory sits on the latency of a step.
//   * K and V stages are TMA boxes (64 columns x 16 rows, never across a page)
//     with the 128-byte swizzle, read back by ldmatrix without bank conflicts.
//   * P = 2^(s - m) is rounded to the cache's type for the second product (its
//     matrix instruction has one input type); sums use the unrounded value.
//     The reference m is the maximum of a row's first keys and moves only when P
//     passes 2^15.  In fp16 P is scaled by 2^7, so probabilities down to 2^-21
//     stay normal.
//   * keys behind a sequence's length: scores are replaced before they are
//     used, V rows are zeroed in shared memory, so whatever the page holds
//     there (NaN included) cannot reach the result.
#pragma once
#include <cuda.h>
#include <limits.h>

#include "paged_sched.cuh"

namespace s2o {

constexpr int kPgKeys = 64;                        // keys of a unit
constexpr int kPgSub = 16;                         // keys of a stage
constexpr uint32_t kPgStage = 2 * kPgSub * 256;    // K then V, each two halves of 16 rows x 128 bytes
constexpr int kPgWarps = 8;
constexpr float kPgScale = 1.4426950408889634f * 0.08838834764831845f;  // log2(e) / sqrt(128)
// A row's reference is the maximum of the first keys it saw.  Later ones need
// no maximum: numbers with an exponent lose nothing by being large, so the
// reference moves only when P passes 2^15: in fp16 the type's end, in bf16 room
// enough for the accumulator below fp32's.
constexpr float kPgMove = 32768.f;

template <int R>
struct PgDecode {
  static constexpr int kStreams = kPgWarps / R;
  static constexpr int kStages = 3 * R;            // of a stream; 24 in all
  static constexpr int kPieces = 4 * R;            // piece slots of a stream: more than stages
  static constexpr uint32_t kOffPiece = kStreams * kStages * kPgStage;
  static constexpr uint32_t kOffBar = kOffPiece + kStreams * kPieces * 64;
  static constexpr int kBars = 2 * kStages;        // of a stream: full, empty
  static constexpr uint32_t kOffRed = kOffBar + kStreams * kBars * 8;
  static constexpr uint32_t kBytes = kOffRed + 34 * 8 + kPgWarps * sizeof(SchedFound);
  static constexpr size_t kSmem = kBytes + 1024;
};

// Unfinished rows: fp32 accumulators and (reference, sum), base-2 exponents.
// A row's columns stand in the order of the accumulator fragments: of every 32,
// place 8 q + 2 j + e has column 8 j + 2 q + e (j, q < 4, e < 2), so that the
// four threads of a fragment's row write its 32 columns as one line.
struct PagedPart {
  float* dense[2];      // [Tq * Hq, 128]: rows of items that one share holds whole (0: prefix, 1: own)
  float2* dense_ml[2];  // [Tq * Hq]
  float* slots;      // [2 workers, rows, 128]
  float2* slots_ml;  // [2 workers, rows]
  int rows;          // rows of a slot
};

// what a kernel tells the join: its units and its workers
struct PagedHead {
  int64_t units;
  int64_t workers;
};

struct PagedArgs {
  PagedGeom g;
  PagedCut c;
  PagedCut other;     // side by side: the other kernel's
  const uint16_t* Q;  // [Tq, Hq, 128]
  void* O;
  float* lse;         // [Tq, Hq] or null
  PagedPart part;
  // where the join finds the parts of own items, one of the two:
  int4* meta;         // [Tq, Hkv]: first and last share of the token's item, its place in the tile
  SplitItem* split;   // [workers]: the item that begins in a share and goes on
  PagedHead* head;
  int out_f32;
  int direct;         // whole items are the result (no other list of keys to join)
  int beside;         // tile and decode kernel share the SMs
  float own_ns;       // see decode_sms
};

// the outcome of a wait that every lane made, agreed on by the warp
__device__ __forceinline__ bool warp_ok(bool ok) { return __all_sync(0xffffffffu, ok); }

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <bool FP16>
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if (FP16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void tma_load_rows(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar,
                                              uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1, {%2, %3}], [%4], %5;\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "l"(policy)
      : "memory");
}
// L2 policies.  Keys that one worker (or one team, at about the same time) reads
// go first when L2 is full: they leave the kernels' code and the parts there.
// Fetched from memory, the code alone held every CTA up for 8 us (64 sequences
// of up to 1023 keys behind 32K: 85.5 us a pass with no hint, 75.8 so).  Keys
// that several items read stay as long as others (five prompt chunks of up to
// 1023 tokens behind 8K: 440 us; 505 if theirs go first, too).
__device__ __forceinline__ uint64_t keys_policy(bool once) {
  uint64_t first, normal;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;\n" : "=l"(first));
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;\n" : "=l"(normal));
  return once ? first : normal;
}
// Programmatic launch: the kernel behind this one may start on SMs that this
// one leaves; and the wait until the kernel in front is done and its writes
// are seen (both nothing when the launch did not ask for it).
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }
// the tensor map on its way before the first copy asks for it
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
// two neighbouring values of a finished row
template <bool FP16>
__device__ __forceinline__ void store2(void* O, int out_f32, size_t at, float x, float y) {
  if (out_f32) *reinterpret_cast<float2*>(static_cast<float*>(O) + at) = make_float2(x, y);
  else *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(O) + at) = pack2<FP16>(x, y);
}
// thread q's eight columns of 32 of an unfinished row (see PagedPart)
__device__ __forceinline__ void store_part(float* block, int q, float v0, float v1, float v2, float v3, float v4,
                                           float v5, float v6, float v7) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(block + 8 * q), "f"(v0), "f"(v1),
               "f"(v2), "f"(v3), "f"(v4), "f"(v5), "f"(v6), "f"(v7)
               : "memory");
}
__device__ __forceinline__ float lse_of(float ref, float sum) {
  return sum == 0.f ? -INFINITY : (ref + log2f(sum)) * 0.6931471805599453f;
}

// A piece's keys are at most two runs of a page list: the prefix's tiles, then
// the sequence's own.  Run k (0 prefix, 1 own) in 16-key parts; `len` keys of
// the list can be reached by the rows.
struct KeyRun {
  int sub0, sub1, len;
};
__device__ __forceinline__ KeyRun key_run(const PagedGeom& g, const Piece& p, int k) {
  KeyRun r;
  const bool pre = p.kind == 0;
  const int t0 = k == 0 ? p.tile0 : (pre ? 0 : max(p.tile0 - p.np, 0));
  const int t1 = k == 0 ? (pre ? p.tile1 : min(p.tile1, p.np)) : (pre ? 0 : p.tile1 - p.np);
  r.len = k == 0 ? g.prefix : p.len;
  r.sub0 = t0 * (kPgKeys / kPgSub);
  r.sub1 = t1 > t0 ? (min(r.len, t1 * kPgKeys) + kPgSub - 1) / kPgSub : r.sub0;
  return r;
}

// the page of a box of keys: clamped and flagged when it is none of the cache's
__device__ __forceinline__ int checked_page(const PagedGeom& g, const int32_t* list, int64_t i) {
  const int p = list[i];
  if (p < 0 || p >= g.num_pages) {
    set_error(kErrBadCache);
    return 0;
  }
  return p;
}

// Tells the join where the rows of an own item are: per token, or (chunks, whose
// rows are many and whose items are seldom split) one record a share, written
// at its end.
__device__ __forceinline__ void announce_split(const PagedArgs& a, const Sched& sc, const Piece& p, SplitItem& split,
                                               int lane) {
  if (p.kind == 1 && p.first) {
    const int c1 = p.last ? sc.me : split_end(sc);
    if (a.meta) {
      for (int t = lane; t < p.ntok; t += 32)
        a.meta[(int64_t)(p.tok0 + t) * a.g.Hkv + p.kvh] = make_int4(sc.me, c1, t, 0);
    } else if (!p.last) {
      split = {p.tok0, p.ntok, p.kvh, c1};
    }
  }
  if (p.kind < 0 && a.split && lane == 0) a.split[sc.me] = split;
}

template <bool FP16, int R>
__global__ void __launch_bounds__(32 * kPgWarps, 1)
    k_paged_decode(const __grid_constant__ PagedArgs a, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV) {
  using C = PgDecode<R>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* sgen = smem_raw + (sbase - smem_u32(smem_raw));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int stream = warp / R, rt = warp % R;
  const uint32_t ring = sbase + stream * C::kStages * kPgStage;
  const uint32_t bars = sbase + C::kOffBar + stream * C::kBars * 8;
  auto full = [&](int st) { return bars + 8u * st; };
  auto empty = [&](int st) { return bars + 8u * (C::kStages + st); };
  auto piece_at = [&](uint32_t k) {
    return reinterpret_cast<Piece*>(sgen + C::kOffPiece + (stream * C::kPieces + k % C::kPieces) * 64);
  };
  static_assert(sizeof(Piece) <= 64, "piece slot");
  const PagedGeom& g = a.g;
  let_next_start();

  if (tid == 0) {
    prefetch_map(&tmK);
    prefetch_map(&tmV);
  }
  if (rt == 0 && lane < C::kStages) {
    mbar_init(full(lane), 1);
    mbar_init(empty(lane), R);
    fence_mbar_init();
  }
  SchedFound* found = reinterpret_cast<SchedFound*>(sgen + C::kOffRed + 34 * 8);
  const OwnRun run = own_run(g, a.c, C::kStreams, reinterpret_cast<int64_t*>(sgen + C::kOffRed), found);
  const int ctas = a.beside ? decode_sms(g, a.other, batch_tokens(g), run.total, a.own_ns, gridDim.x) : (int)gridDim.x;
  Sched sc = sched_begin(g, a.c, C::kStreams, stream, ctas, run, found);
  if (tid == 0 && blockIdx.x == 0) *a.head = {sc.U, ctas * C::kStreams};
  __syncthreads();

  // ---- the stream's loads, by its first warp: stage by stage through the
  // pieces.  A piece's description goes into its slot before the arrival on its
  // first stage; the end is a piece of kind -1 with a stage that loads nothing.
  // A piece holds at least one stage, so a slot is read before it comes round.
  uint32_t put = 0, pieces_put = 0;     // stages and pieces announced
  int sub = 0, sub1 = 0, base = 0;      // next and last 16 keys of the run; first of the lanes' pages
  int page = 0, page_next = 0;          // page of 16 keys base + lane, and of the 32 behind
  int keys = 1;                         // run of the piece
  Piece ip;
  ip.kind = 0;
  const int32_t* list = nullptr;
  SplitItem split = {0, 0, 0, 0};
  const int sub_log2 = g.page_log2 - 4;  // 16-key parts of a page
  const uint64_t own_policy = keys_policy(true), prefix_policy = keys_policy(false);
  bool ok = true;
  auto issue = [&]() {
    if (ip.kind < 0) return;
    const int st = put % C::kStages;
    if (R > 1) {  // the other warps have read what was there
      if (!warp_ok(mbar_wait_bounded(empty(st), ((put / C::kStages) & 1) ^ 1))) {
        ok = false;
        return;
      }
    }
    while (sub == sub1) {  // the next run, of this piece or the next
      if (++keys == 2) {
        ip = sched_next(g, a.c, sc);
        if (lane == 0) *piece_at(pieces_put) = ip;
        ++pieces_put;
        announce_split(a, sc, ip, split, lane);
        if (ip.kind < 0) {
          __syncwarp();
          if (lane == 0) mbar_arrive(full(st));
          ++put;
          return;
        }
        keys = 0;
      }
      const KeyRun r = key_run(g, ip, keys);
      list = keys == 0 ? g.prefix_pages : g.table + (int64_t)ip.seq * g.max_pages;
      sub = base = r.sub0;
      sub1 = r.sub1;
      page = sub + lane < sub1 ? checked_page(g, list, (sub + lane) >> sub_log2) : 0;
      page_next = sub + 32 + lane < sub1 ? checked_page(g, list, (sub + 32 + lane) >> sub_log2) : 0;
    }
    if (sub - base == 32) {
      page = page_next;
      base = sub;
      page_next = sub + 32 + lane < sub1 ? checked_page(g, list, (sub + 32 + lane) >> sub_log2) : 0;
    }
    const int pg = __shfl_sync(0xffffffffu, page, sub - base);
    if (lane == 0) mbar_expect_tx(full(st), kPgStage);
    __syncwarp();
    if (lane < 4) {
      const int half = lane & 1, isv = lane >> 1;
      const int y = ((pg * g.Hkv + ip.kvh) << g.page_log2) + ((sub & ((1 << sub_log2) - 1)) << 4);
      tma_load_rows(ring + st * kPgStage + isv * (kPgSub * 256) + half * (kPgSub * 128), isv ? &tmV : &tmK, 64 * half,
                    y, full(st), keys == 1 ? own_policy : prefix_policy);
    }
    ++sub;
    ++put;
  };
  if (rt == 0)
    for (int k = 0; k < C::kStages && ok; ++k) issue();

  // ---- the rows
  const int r0 = lane >> 2, cq = 2 * (lane & 3);
  constexpr float kShift = FP16 ? 7.f : 0.f;
  uint32_t it = 0;
  for (uint32_t pi = 0; ok; ++pi) {
    if (!warp_ok(mbar_wait_bounded(full(it % C::kStages), (it / C::kStages) & 1))) { ok = false; break; }
    const Piece p = *piece_at(pi);
    if (p.kind < 0) break;
    const int rows = p.ntok * g.G;
    const bool active = 16 * rt < rows;
    // this lane's rows: r0 and r0 + 8 of the warp's 16
    int lim_own[2];   // own keys < lim_own are seen
    size_t orow[2];   // row of [Tq, Hq]
    bool has[2];
    uint32_t qf[8][4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int r = 16 * rt + r0 + 8 * k;
      has[k] = r < rows;
      const int tt = has[k] ? r / g.G : 0, h = has[k] ? r - tt * g.G : 0;
      lim_own[k] = has[k] ? p.off + tt + 1 : INT_MAX;  // rows of nobody see everything: no masks for their sake
      orow[k] = (size_t)(p.tok0 + tt) * g.Hq + p.kvh * g.G + h;
      const uint16_t* q = a.Q + orow[k] * kD + cq;
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        qf[kk][k] = has[k] ? *reinterpret_cast<const uint32_t*>(q + 16 * kk) : 0u;
        qf[kk][k + 2] = has[k] ? *reinterpret_cast<const uint32_t*>(q + 16 * kk + 8) : 0u;
      }
    }
    float acc[16][4];
#pragma unroll
    for (int n = 0; n < 16; ++n)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[n][k] = 0.f;
    float ref[2] = {0.f, 0.f}, sum[2] = {0.f, 0.f};
    bool fresh = true;  // the references are still to be set

    for (int keys = 0; keys < 2; ++keys) {
    const KeyRun r = key_run(g, p, keys);
    const int lim[2] = {keys == 0 ? r.len : lim_own[0], keys == 0 ? r.len : lim_own[1]};
    // the fewest keys that a row of the warp sees
    const int lim_min = __reduce_min_sync(0xffffffffu, min(lim[0], lim[1]));
    for (int t = r.sub0; t < r.sub1; ++t, ++it) {
      const int st = it % C::kStages;
      if (!warp_ok(mbar_wait_bounded(full(st), (it / C::kStages) & 1))) { ok = false; break; }
      if (active) {
        const int key0 = t * kPgSub;
        const uint32_t sK = ring + st * kPgStage, sV = sK + kPgSub * 256;
        float x[2][4] = {}, y[2][4] = {};  // two chains of products each
        {
          const uint32_t row = (lane & 7) + 8 * (lane >> 4);
#pragma unroll
          for (int kk = 0; kk < 8; kk += 2) {
            uint32_t b[4], c[4];
            ldsm4(sK + (kk >> 2) * (kPgSub * 128) + swz128(row, 2 * (kk & 3) + ((lane >> 3) & 1)), b);
            ldsm4(sK + (kk >> 2) * (kPgSub * 128) + swz128(row, 2 * (kk & 3) + 2 + ((lane >> 3) & 1)), c);
            mma16816<FP16>(x[0], qf[kk], b[0], b[1]);
            mma16816<FP16>(x[1], qf[kk], b[2], b[3]);
            mma16816<FP16>(y[0], qf[kk + 1], c[0], c[1]);
            mma16816<FP16>(y[1], qf[kk + 1], c[2], c[3]);
          }
        }
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) x[n][k] += y[n][k];
        if (key0 + kPgSub > lim_min) {  // hidden keys
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (key0 + 8 * n + cq + (k & 1) >= lim[k >> 1]) x[n][k] = -INFINITY;
        }
        float px[2][4];
        auto exponentials = [&]() {
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int k = 0; k < 4; ++k) px[n][k] = ex2_approx(fmaf(x[n][k], kPgScale, -ref[k >> 1]));
        };
        bool move = fresh;
        if (!fresh) {
          exponentials();
          const float top = fmaxf(fmaxf(fmaxf(px[0][0], px[0][1]), fmaxf(px[0][2], px[0][3])),
                                  fmaxf(fmaxf(px[1][0], px[1][1]), fmaxf(px[1][2], px[1][3])));
          move = __any_sync(0xffffffffu, top > kPgMove);
        }
        if (move) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float mx = fmaxf(fmaxf(x[0][2 * k], x[0][2 * k + 1]), fmaxf(x[1][2 * k], x[1][2 * k + 1]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            mx = fmaf(mx, kPgScale, -kShift);
            if (fresh) {
              ref[k] = mx == -INFINITY ? 0.f : mx;  // sees nothing here, and nothing behind it
            } else if (mx > ref[k]) {
              const float f = ex2_approx(ref[k] - mx);
              ref[k] = mx;
              sum[k] *= f;
#pragma unroll
              for (int n = 0; n < 16; ++n) {
                acc[n][2 * k] *= f;
                acc[n][2 * k + 1] *= f;
              }
            }
          }
          fresh = false;
          exponentials();
        }
        uint32_t pf[4];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          sum[0] += px[n][0] + px[n][1];
          sum[1] += px[n][2] + px[n][3];
          pf[2 * n] = pack2<FP16>(px[n][0], px[n][1]);
          pf[2 * n + 1] = pack2<FP16>(px[n][2], px[n][3]);
        }
        if (key0 + kPgSub > r.len) {
          // V rows behind the list: zero (the stream's other warps write the
          // same zeros); before the stage's next TMA write, a proxy fence
          for (int i = lane; i < kPgSub * 16; i += 32) {
            const int row = i >> 4, ch = i & 15;
            if (key0 + row >= r.len)
              *reinterpret_cast<uint4*>(sgen + (sV - sbase) + (ch >> 3) * (kPgSub * 128) + swz128(row, ch & 7)) =
                  make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        {
          const uint32_t row = (lane & 7) + 8 * ((lane >> 3) & 1);
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            uint32_t b[4];
            const uint32_t ch = 2 * n + (lane >> 4);
            ldsm4_t(sV + (n >> 2) * (kPgSub * 128) + swz128(row, ch & 7), b);
            mma16816<FP16>(acc[2 * n], pf, b[0], b[1]);
            mma16816<FP16>(acc[2 * n + 1], pf, b[2], b[3]);
          }
        }
      }
      __syncwarp();
      if (R > 1 && lane == 0) mbar_arrive(empty(st));
      // the next load into the stage just read; with other warps at it, into
      // the one before, which they have left by now
      if (rt == 0 && (R == 1 || it > 0)) issue();
      if (!ok) break;
    }
    if (!ok) break;
    }
    if (!ok) break;
    if (!active) continue;

#pragma unroll
    for (int k = 0; k < 2; ++k) {
      sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 1);
      sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 2);
      if (sum[k] == 0.f) ref[k] = -INFINITY;  // saw no key
    }
    const bool whole = p.first && p.last;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (!has[k]) continue;
      if (whole && a.direct) {
        const float inv = sum[k] == 0.f ? 0.f : 1.f / sum[k];
#pragma unroll
        for (int n = 0; n < 16; ++n)
          store2<FP16>(a.O, a.out_f32, orow[k] * kD + 8 * n + cq, acc[n][2 * k] * inv, acc[n][2 * k + 1] * inv);
        if (a.lse && (lane & 3) == 0) a.lse[orow[k]] = lse_of(ref[k], sum[k]);
        continue;
      }
      const size_t at =
          whole ? orow[k] : (size_t)(2 * p.share + (p.first ? 1 : 0)) * a.part.rows + 16 * rt + r0 + 8 * k;
      float* dst = (whole ? a.part.dense[p.kind] : a.part.slots) + at * kD;
#pragma unroll
      for (int n = 0; n < 16; n += 4)
        store_part(dst + 8 * n, lane & 3, acc[n][2 * k], acc[n][2 * k + 1], acc[n + 1][2 * k], acc[n + 1][2 * k + 1],
                   acc[n + 2][2 * k], acc[n + 2][2 * k + 1], acc[n + 3][2 * k], acc[n + 3][2 * k + 1]);
      if ((lane & 3) == 0) (whole ? a.part.dense_ml[p.kind] : a.part.slots_ml)[at] = make_float2(ref[k], sum[k]);
    }
  }
  if (!ok && lane == 0) {
    set_error(kErrTimeout);
  }
  // nothing may land in shared memory after the CTA ends
  if (rt == 0)
    for (uint32_t k = put > (uint32_t)C::kStages ? put - C::kStages : 0; k < put; ++k)
      if (!mbar_wait_bounded(full(k % C::kStages), (k / C::kStages) & 1)) {
        if (lane == 0) set_error(kErrTimeout);
      }
  // nothing here reads what the kernel in front wrote, but the join, which
  // waits for this one alone, does
  wait_for_previous();
}

// ---------------------------------------------------------------------------
// The join: a warp per query row adds the row's parts (the prefix's, then the
// own keys', each in share order, so the result does not depend on timing).  The
// lanes take the (reference, sum) of up to 32 parts at once, agree on the
// common reference and the weights, then read the accumulators with
// independent loads: read one by one, each part costs a trip to L2 (23 to 29 us
// for 2048 rows of 20 parts that take 9 so).

struct JoinSide {
  PagedPart part;
  PagedCut c;
  const PagedHead* head;  // of the kernel that wrote it
  int n;              // its workers at most
};

struct JoinArgs {
  PagedGeom g;
  JoinSide prefix, own;
  const int4* meta;
  const SplitItem* split;
  void* O;
  float* lse;
  int out_f32;
  int direct;         // no prefix items, and what was not split is the result
};

struct RowSum {
  float m, l;
  float4 o;
};
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float warp_add(float x) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
// cnt parts; lane l of a batch of 32 gets part l's (reference, sum) and
// accumulators from part(j, acc); one that saw no key has (-inf, 0).  B loads
// of accumulators are in flight at a time.
template <int B, class F>
__device__ __forceinline__ void add_parts(RowSum& s, int cnt, int lane, F part) {
  for (int base = 0; base < cnt; base += 32) {
    const float* acc = nullptr;
    float2 ml = make_float2(-INFINITY, 0.f);
    if (base + lane < cnt) ml = part(base + lane, acc);
    const float m = fmaxf(s.m, warp_max(ml.x));
    const float w = ml.x == -INFINITY && ml.y == 0.f ? 0.f : ex2_approx(ml.x - m);
    const float f = s.m == -INFINITY ? 0.f : ex2_approx(s.m - m);
    s.m = m;
    s.l = s.l * f + warp_add(ml.y * w);
    s.o = make_float4(s.o.x * f, s.o.y * f, s.o.z * f, s.o.w * f);
    const int n = min(32, cnt - base);
    for (int k0 = 0; k0 < n; k0 += B) {
      float4 v[B];
      float wk[B];
#pragma unroll
      for (int k = 0; k < B; ++k) {
        wk[k] = __shfl_sync(0xffffffffu, w, k0 + k);
        const float4* a = reinterpret_cast<const float4*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(acc), k0 + k));
        v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (wk[k] != 0.f) v[k] = a[lane];  // lanes behind the last part have weight 0
      }
#pragma unroll
      for (int k = 0; k < B; ++k)
        s.o = make_float4(fmaf(v[k].x, wk[k], s.o.x), fmaf(v[k].y, wk[k], s.o.y), fmaf(v[k].z, wk[k], s.o.z),
                          fmaf(v[k].w, wk[k], s.o.w));
    }
  }
}
// A block's four warps on one row: warp w takes the parts w, w + 4, ... and
// the first adds the four sums, in order.  Few rows have many parts (one for
// each share of their item), and a warp would read them in turns.
constexpr int kJoinWarps = 4;
struct JoinShared {
  float m[kJoinWarps], l[kJoinWarps];
  float4 o[kJoinWarps][32];
};
template <class F>
__device__ __forceinline__ RowSum block_add_parts(JoinShared& sh, int cnt, int warp, int lane, F part) {
  RowSum s = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  add_parts<8>(s, (cnt - warp + kJoinWarps - 1) / kJoinWarps, lane,
               [&](int j, const float*& acc) { return part(kJoinWarps * j + warp, acc); });
  if (lane == 0) {
    sh.m[warp] = s.m;
    sh.l[warp] = s.l;
  }
  sh.o[warp][lane] = s.o;
  __syncthreads();
  if (warp == 0) {
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) m = fmaxf(m, sh.m[w]);
    s = {m, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      const float f = sh.m[w] == -INFINITY && sh.l[w] == 0.f ? 0.f : ex2_approx(sh.m[w] - m);
      const float4 v = sh.o[w][lane];
      s.l = fmaf(sh.l[w], f, s.l);
      if (f != 0.f)
        s.o = make_float4(fmaf(v.x, f, s.o.x), fmaf(v.y, f, s.o.y), fmaf(v.z, f, s.o.z), fmaf(v.w, f, s.o.w));
    }
  }
  return s;
}
// part j of an item in shares c0 .. (member `offset` of teams of `stride`)
__device__ __forceinline__ float2 split_part(const PagedPart& part, int c0, int j, int stride, int offset,
                                             int tile_row, const float*& acc) {
  const size_t at = (size_t)(2 * ((c0 + j) * stride + offset) + (j == 0 ? 1 : 0)) * part.rows + tile_row;
  acc = part.slots + at * kD;
  return part.slots_ml[at];
}
__device__ __forceinline__ float2 dense_part(const PagedPart& part, int kind, size_t row, const float*& acc) {
  acc = part.dense[kind] + row * kD;
  return part.dense_ml[kind][row];
}
template <bool FP16>
__device__ __forceinline__ void finish_row(const JoinArgs& a, const RowSum& s, size_t row, int lane) {
  const float inv = s.l == 0.f ? 0.f : 1.f / s.l;
  // places 4 lane .. + 3 of the parts (see PagedPart)
  const size_t at = row * kD + 32 * (lane >> 3) + 16 * (lane & 1) + 2 * ((lane >> 1) & 3);
  store2<FP16>(a.O, a.out_f32, at, s.o.x * inv, s.o.y * inv);
  store2<FP16>(a.O, a.out_f32, at + 8, s.o.z * inv, s.o.w * inv);
  if (a.lse && lane == 0) a.lse[row] = lse_of(s.m, s.l);
}

// Every row of the batch: its prefix parts and its own.  With MANY rows a warp
// each, which hide each other's trips to memory (64 registers, more warps);
// with few a block each.
template <bool FP16, bool MANY>
__global__ void __launch_bounds__(32 * kJoinWarps, 8) k_paged_join(const __grid_constant__ JoinArgs a) {
  __shared__ JoinShared sh;
  const PagedGeom& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = MANY ? blockIdx.x * kJoinWarps + warp : blockIdx.x;
  const int t = row / g.Hq, h = row - t * g.Hq;
  wait_for_previous();
  if (t >= g.Tq) return;
  const int ntok = batch_tokens(g);
  const int kvh = h / g.G, hh = h - kvh * g.G;
  int4 own = a.meta[(int64_t)t * g.Hkv + kvh];
  const int64_t PU = a.direct ? 0 : a.prefix.head->units;
  const int64_t PW = a.direct ? 0 : a.prefix.head->workers;
  if (t >= ntok) return;
  own.x = max(0, min(own.x, a.own.n - 1));  // rows of a refused sequence were never written
  own.y = max(own.x, min(own.y, a.own.n - 1));
  own.z = max(0, min(own.z, a.own.c.tpt - 1));
  int parts = 0, c0 = 0, team = 1, member = 0, prow = 0;
  if (!a.direct) {
    const PagedCut& c = a.prefix.c;
    const int npt = (ntok + c.tpt - 1) / c.tpt, rt = t / c.tpt;
    const int64_t np = prefix_units(g.prefix, c);
    const int workers = max(1, min((int)PW, a.prefix.n));
    team = team_size(c, npt, workers);
    const int n = shares_of(PU, workers / team);
    const int64_t u0 = (team > 1 ? (int64_t)kvh : (int64_t)kvh * npt + rt) * np;
    c0 = share_owner(PU, n, u0 + c.fixed);  // of the first keys
    parts = share_owner(PU, n, u0 + np - 1) - c0 + 1;
    member = team > 1 ? rt : 0;
    prow = (t - rt * c.tpt) * g.G + hh;
  } else if (own.x == own.y) {
    return;
  }
  auto part = [&](int j, const float*& acc) {
    if (j < parts)
      return parts == 1 ? dense_part(a.prefix.part, 0, row, acc)
                        : split_part(a.prefix.part, c0, j, team, member, prow, acc);
    return own.x == own.y ? dense_part(a.own.part, 1, row, acc)
                          : split_part(a.own.part, own.x, j - parts, 1, 0, own.z * g.G + hh, acc);
  };
  const int cnt = parts + own.y - own.x + 1;
  RowSum s = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  if constexpr (MANY) add_parts<4>(s, cnt, lane, part);
  else s = block_add_parts(sh, cnt, warp, lane, part);
  if (MANY || warp == 0) finish_row<FP16>(a, s, row, lane);
}

// chunks: own items that two or more workers share (all others are the result
// already); block (c, y) takes every gridDim.y-th four rows of the one that
// begins in share c and goes on, a warp each
template <bool FP16>
__global__ void __launch_bounds__(32 * kJoinWarps) k_paged_join_split(const __grid_constant__ JoinArgs a) {
  const PagedGeom& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  wait_for_previous();
  const SplitItem it = a.split[blockIdx.x];
  for (int r = blockIdx.y * kJoinWarps + warp; r < it.ntok * g.G; r += gridDim.y * kJoinWarps) {
    const int t = r / g.G;
    RowSum s = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    add_parts<8>(s, it.c1 - (int)blockIdx.x + 1, lane,
                 [&](int j, const float*& acc) { return split_part(a.own.part, blockIdx.x, j, 1, 0, r, acc); });
    finish_row<FP16>(a, s, (size_t)(it.tok0 + t) * g.Hq + it.kvh * g.G + (r - t * g.G), lane);
  }
}

}  // namespace s2o
