// Attention over a paged cache, few query rows a KV head: one token or a few
// drafted ones of every sequence (the sequences' own keys), and a shared
// prefix when the whole batch is few rows.
//
//   o_i = sum_j exp(s_ij) v_j / sum_j exp(s_ij),  s_ij = q_i . k_j / sqrt(d),
//   j over the prefix and the own keys up to the row's own
//
// Bound by the cache: a key and its value are 512 bytes for 4 d flops a row,
// 16 flops a byte at 16 rows, far below what the GPU can do, so the kernel is
// built to keep reads in flight: one CTA per SM, a producer warp that fills a
// ring of 64-key stages (32 KB each) with TMA tiles of the pages' rows, and
// consumer warps that turn a stage around in a fraction of the time HBM needs
// for it.
//
//   * warps: R row tiles of 16 rows (an mma's M) x 4 key slices of 16 keys; a
//     warp holds its own running reference and sum and a 16 x 128 fp32
//     accumulator in registers, so a stage needs no exchange between warps;
//     the four slices are joined once per piece, through shared memory.
//   * products: mma.sync m16n8k16 (bf16 or fp16 in, fp32 out).  With at most
//     64 rows a KV head the 128-row tcgen05 tile would be mostly empty and
//     its round trip through tensor memory sits on the latency of a step.
//   * K and V tiles are TMA boxes (64 columns x min(page, 64) rows) with the
//     128-byte swizzle, read back by ldmatrix without bank conflicts.
//   * P = 2^(s - m) is rounded to the cache's type for the second product (its
//     matrix instruction has one input type); sums use the unrounded value.
//     The reference m moves only when the maximum grows by more than 2^8.  In
//     fp16 P is scaled by 2^7, so probabilities down to 2^-21 stay normal.
//   * keys behind a sequence's length: scores are replaced before they are
//     used, V rows are zeroed in shared memory, so whatever the page holds
//     there (NaN included) cannot reach the result.
#pragma once
#include <cuda.h>

#include "paged_sched.cuh"

namespace s2o {

constexpr int kPgKeys = 64;                        // keys of a stage
constexpr uint32_t kPgStage = 2 * kPgKeys * 256;   // K then V
constexpr int kPieceSlots = 4;
constexpr float kPgScale = 1.4426950408889634f * 0.08838834764831845f;  // log2(e) / sqrt(128)

template <int R>
struct PgDecode {
  static constexpr int kThreads = 128 * R + 32;
  static constexpr int kStages = R == 4 ? 4 : (R == 2 ? 5 : 6);
  static constexpr uint32_t kOffJoin = kStages * kPgStage;              // [R][2][16][kJoinPitch] fp32
  static constexpr uint32_t kJoinPitch = 132;
  static constexpr uint32_t kOffMl = kOffJoin + R * 2 * 16 * kJoinPitch * 4;  // [R][4][16] float2
  static constexpr uint32_t kOffPiece = kOffMl + R * 4 * 16 * 8;
  static constexpr uint32_t kOffBar = kOffPiece + kPieceSlots * 64;
  static constexpr int kBarFull = 0, kBarEmpty = kStages, kBarPieceFull = 2 * kStages,
                       kBarPieceEmpty = 2 * kStages + kPieceSlots, kBarJoin = 2 * kStages + 2 * kPieceSlots,
                       kBars = kBarJoin + R;
  static constexpr uint32_t kOffRed = kOffBar + 8 * ((kBars + 1) & ~1);
  static constexpr uint32_t kBytes = kOffRed + 34 * 8 + 16;
  static constexpr size_t kSmem = kBytes + 1024;
};

// Unfinished rows: fp32 accumulators and (reference, sum), base-2 exponents.
struct PagedPart {
  float* dense[2];      // [Tq * Hq, 128]: rows of items that one CTA holds whole (0: prefix, 1: own)
  float2* dense_ml[2];  // [Tq * Hq]
  float* slots;      // [2 n, rows, 128]
  float2* slots_ml;  // [2 n, rows]
  int rows;          // rows of a slot
};

struct PagedArgs {
  PagedGeom g;
  PagedCut c;
  const uint16_t* Q;  // [Tq, Hq, 128]
  void* O;
  float* lse;         // [Tq, Hq] or null
  PagedPart part;
  int2* meta;         // [Tq, Hkv]: CTAs of the own item a token's rows are in
  int64_t* units;     // total units of this kernel, for the join
  int out_f32;
  int direct;         // whole items are the result (no other list of keys to join)
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
__device__ __forceinline__ void tma_load_rows(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
// two neighbouring values of a finished row
template <bool FP16>
__device__ __forceinline__ void store2(void* O, int out_f32, size_t at, float x, float y) {
  if (out_f32) *reinterpret_cast<float2*>(static_cast<float*>(O) + at) = make_float2(x, y);
  else *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(O) + at) = pack2<FP16>(x, y);
}
__device__ __forceinline__ float lse_of(float ref, float sum) {
  return sum == 0.f ? -INFINITY : (ref + log2f(sum)) * 0.6931471805599453f;
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

template <bool FP16, int R>
__global__ void __launch_bounds__(PgDecode<R>::kThreads, 1)
    k_paged_decode(const __grid_constant__ PagedArgs a, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV) {
  using C = PgDecode<R>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* sgen = smem_raw + (sbase - smem_u32(smem_raw));
  auto bar = [&](int k) { return sbase + C::kOffBar + 8u * (uint32_t)k; };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const PagedGeom& g = a.g;

  if (tid == 0) {
    for (int k = 0; k < C::kStages; ++k) {
      mbar_init(bar(C::kBarFull + k), 1);
      mbar_init(bar(C::kBarEmpty + k), 4 * R);
    }
    for (int k = 0; k < kPieceSlots; ++k) {
      mbar_init(bar(C::kBarPieceFull + k), 1);
      mbar_init(bar(C::kBarPieceEmpty + k), 4 * R);
    }
    for (int k = 0; k < R; ++k) mbar_init(bar(C::kBarJoin + k), 4);
    fence_mbar_init();
  }
  Sched sc = sched_begin(g, a.c, reinterpret_cast<int64_t*>(sgen + C::kOffRed),
                         reinterpret_cast<SchedFound*>(sgen + C::kOffRed + 33 * 8));
  if (tid == 0 && blockIdx.x == 0) *a.units = sc.U;
  __syncthreads();
  static_assert(sizeof(Piece) <= 64, "piece slot");
  auto piece_at = [&](int k) { return reinterpret_cast<Piece*>(sgen + C::kOffPiece + 64 * k); };

  if (warp == 4 * R) {
    // ------------------------------------------------------------------ producer
    const int box_log2 = min(g.page_log2, 6);              // rows of a box
    const int boxes = kPgKeys >> box_log2;                 // of a full stage
    const int rest_log2 = g.page_log2 - box_log2;          // boxes of a page
    bool ok = true;
    uint32_t it = 0;
    for (int pi = 0; ok; ++pi) {
      const Piece p = sched_next(g, a.c, sc);
      const int slot = pi % kPieceSlots;
      if (!warp_ok(mbar_wait_bounded(bar(C::kBarPieceEmpty + slot), ((pi / kPieceSlots) & 1) ^ 1))) { ok = false; break; }
      if (lane == 0) {
        *piece_at(slot) = p;
        mbar_arrive(bar(C::kBarPieceFull + slot));
      }
      if (p.kind < 0) break;
      if (p.kind == 1 && p.first)  // where the join finds the rows of this item
        for (int t = lane; t < p.ntok; t += 32) a.meta[(int64_t)(p.tok0 + t) * g.Hkv + p.kvh] = make_int2(p.c0, p.c1);
      const int32_t* list = p.kind == 0 ? g.prefix_pages : g.table + (int64_t)p.seq * g.max_pages;
      // boxes of the piece, taken 32 at a time: a lane holds the page of one
      const int box0 = p.tile0 * boxes, box1 = min(p.tile1 * boxes, (p.len + (1 << box_log2) - 1) >> box_log2);
      int page = 0, page_next = 0;
      if (box0 + lane < box1) page_next = checked_page(g, list, (box0 + lane) >> rest_log2);
      for (int tile = p.tile0; tile < p.tile1; ++tile) {
        const int b0 = tile * boxes, in32 = (b0 - box0) & 31;
        if (in32 == 0) {
          page = page_next;
          const int nb = b0 + 32 + lane;
          if (nb < box1) page_next = checked_page(g, list, nb >> rest_log2);
        }
        const int st = it % C::kStages;
        if (!warp_ok(mbar_wait_bounded(bar(C::kBarEmpty + st), ((it / C::kStages) & 1) ^ 1))) { ok = false; break; }
        const int nb = min(boxes, box1 - b0);
        if (lane == 0) mbar_expect_tx(bar(C::kBarFull + st), (uint32_t)nb << (box_log2 + 9));
        __syncwarp();
        const int i = lane >> 2, half = lane & 1, isv = (lane >> 1) & 1;
        const int pg = __shfl_sync(0xffffffffu, page, (in32 + i) & 31);
        if (i < nb) {
          const int in_page = ((b0 + i) & ((1 << rest_log2) - 1)) << box_log2;
          const int y = (((pg * g.Hkv + p.kvh) << g.page_log2) + in_page);
          tma_load_rows(sbase + st * kPgStage + isv * (kPgKeys * 256) + half * (kPgKeys * 128) + ((i << box_log2) * 128),
                        isv ? &tmV : &tmK, 64 * half, y, bar(C::kBarFull + st));
        }
        ++it;
      }
    }
    if (!ok && lane == 0) set_error(kErrTimeout);
    // nothing may land in shared memory after the CTA ends
    const uint32_t first = it > (uint32_t)C::kStages ? it - C::kStages : 0;
    for (uint32_t k = first; k < it; ++k)
      if (!mbar_wait_bounded(bar(C::kBarFull + k % C::kStages), (k / C::kStages) & 1)) {
        if (lane == 0) set_error(kErrTimeout);
      }
    return;
  }

  // -------------------------------------------------------------------- consumers
  const int rt = warp >> 2, ks = warp & 3;
  const int r0 = lane >> 2, cq = 2 * (lane & 3);
  float* join = reinterpret_cast<float*>(sgen + C::kOffJoin) + rt * (2 * 16 * C::kJoinPitch);
  float2* mls = reinterpret_cast<float2*>(sgen + C::kOffMl) + rt * 64;
  constexpr float kShift = FP16 ? 7.f : 0.f;
  uint32_t it = 0, jphase = 0;
  bool ok = true;
  for (int pi = 0;; ++pi) {
    const int slot = pi % kPieceSlots;
    if (!warp_ok(mbar_wait_bounded(bar(C::kBarPieceFull + slot), (pi / kPieceSlots) & 1))) { ok = false; break; }
    const Piece p = *piece_at(slot);
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(C::kBarPieceEmpty + slot));
    if (p.kind < 0) break;
    const int rows = p.ntok * g.G;
    if (16 * rt >= rows) {  // no rows: let the stages pass
      for (int tile = p.tile0; ok && tile < p.tile1; ++tile, ++it) {
        const int st = it % C::kStages;
        ok = warp_ok(mbar_wait_bounded(bar(C::kBarFull + st), (it / C::kStages) & 1));
        if (ok && lane == 0) mbar_arrive(bar(C::kBarEmpty + st));
      }
      if (!ok) break;
      continue;
    }
    // this lane's rows: r0 and r0 + 8 of the tile
    int lim[2];       // keys < lim are seen
    size_t orow[2];   // row of [Tq, Hq]
    bool has[2];
    uint32_t qf[8][4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int r = 16 * rt + r0 + 8 * k;
      has[k] = r < rows;
      const int tt = has[k] ? r / g.G : 0, h = has[k] ? r - tt * g.G : 0;
      lim[k] = !has[k] ? 0 : (p.kind == 0 ? p.len : p.off + tt + 1);
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
    float ref[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};

    for (int tile = p.tile0; tile < p.tile1; ++tile, ++it) {
      const int st = it % C::kStages;
      if (!warp_ok(mbar_wait_bounded(bar(C::kBarFull + st), (it / C::kStages) & 1))) { ok = false; break; }
      const int key0 = tile * kPgKeys + 16 * ks;
      bool wrote = false;
      if (key0 < p.len) {
        const uint32_t sK = sbase + st * kPgStage, sV = sK + kPgKeys * 256;
        float x[2][4] = {};
        {
          const uint32_t row = 16 * ks + (lane & 7) + 8 * (lane >> 4);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            uint32_t b[4];
            ldsm4(sK + (kk >> 2) * (kPgKeys * 128) + swz128(row, 2 * (kk & 3) + ((lane >> 3) & 1)), b);
            mma16816<FP16>(x[0], qf[kk], b[0], b[1]);
            mma16816<FP16>(x[1], qf[kk], b[2], b[3]);
          }
        }
        // hidden keys, the rows' maxima
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int key = key0 + 8 * n + cq + (k & 1);
            x[n][k] = key < lim[k >> 1] ? x[n][k] * kPgScale : -INFINITY;
            mx[k >> 1] = fmaxf(mx[k >> 1], x[n][k]);
          }
        bool move = false;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], 1));
          mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], 2));
          move |= mx[k] - kShift > ref[k] + 8.f;
        }
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            if (!(mx[k] - kShift > ref[k] + 8.f)) continue;
            const float f = ex2_approx(ref[k] - (mx[k] - kShift));  // ref -inf: 0
            ref[k] = mx[k] - kShift;
            sum[k] *= f;
#pragma unroll
            for (int n = 0; n < 16; ++n) {
              acc[n][2 * k] *= f;
              acc[n][2 * k + 1] *= f;
            }
          }
        }
        uint32_t pf[4];
        {
          const float m0 = ref[0] == -INFINITY ? 0.f : ref[0], m1 = ref[1] == -INFINITY ? 0.f : ref[1];
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const float p0 = ex2_approx(x[n][0] - m0), p1 = ex2_approx(x[n][1] - m0);
            const float p2 = ex2_approx(x[n][2] - m1), p3 = ex2_approx(x[n][3] - m1);
            sum[0] += p0 + p1;
            sum[1] += p2 + p3;
            pf[2 * n] = pack2<FP16>(p0, p1);
            pf[2 * n + 1] = pack2<FP16>(p2, p3);
          }
        }
        if (key0 + 16 > p.len) {
          // V rows behind the list: zero (16-byte chunks; the row tiles' warps
          // of this slice write the same zeros)
          for (int i = lane; i < 16 * 16; i += 32) {
            const int row = i >> 4, ch = i & 15;
            if (key0 + row >= p.len)
              *reinterpret_cast<uint4*>(sgen + (sV - sbase) + (ch >> 3) * (kPgKeys * 128) +
                                        swz128(16 * ks + row, ch & 7)) = make_uint4(0, 0, 0, 0);
          }
          wrote = true;
          __syncwarp();
        }
        {
          const uint32_t row = 16 * ks + (lane & 7) + 8 * ((lane >> 3) & 1);
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            uint32_t b[4];
            const uint32_t ch = 2 * n + (lane >> 4);
            ldsm4_t(sV + (n >> 2) * (kPgKeys * 128) + swz128(row, ch & 7), b);
            mma16816<FP16>(acc[2 * n], pf, b[0], b[1]);
            mma16816<FP16>(acc[2 * n + 1], pf, b[2], b[3]);
          }
        }
      }
      if (wrote) fence_proxy_async_smem();  // before the stage's next TMA write
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::kBarEmpty + st));
    }
    if (!ok) break;

    // ---- the four slices of a row tile become one: sums of the lanes, the
    // common reference, accumulators added pairwise in a fixed order
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 1);
      sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 2);
      if ((lane & 3) == 0) mls[16 * ks + r0 + 8 * k] = make_float2(ref[k], sum[k]);
    }
    auto meet = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::kBarJoin + rt));
      const bool met = warp_ok(mbar_wait_bounded(bar(C::kBarJoin + rt), jphase));
      jphase ^= 1;
      return met;
    };
    if (!meet()) { ok = false; break; }
    float tot[2], top[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float2 v[4];
      top[k] = -INFINITY;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        v[w] = mls[16 * w + r0 + 8 * k];
        top[k] = fmaxf(top[k], v[w].x);
      }
      const float m = top[k] == -INFINITY ? 0.f : top[k];
      tot[k] = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) tot[k] += v[w].y * ex2_approx(v[w].x - m);
      const float f = ex2_approx(ref[k] - m);
#pragma unroll
      for (int n = 0; n < 16; ++n) {
        acc[n][2 * k] *= f;
        acc[n][2 * k + 1] *= f;
      }
    }
    auto put = [&](float* b) {
#pragma unroll
      for (int n = 0; n < 16; ++n) {
        *reinterpret_cast<float2*>(b + r0 * C::kJoinPitch + 8 * n + cq) = make_float2(acc[n][0], acc[n][1]);
        *reinterpret_cast<float2*>(b + (r0 + 8) * C::kJoinPitch + 8 * n + cq) = make_float2(acc[n][2], acc[n][3]);
      }
    };
    auto add = [&](const float* b) {
#pragma unroll
      for (int n = 0; n < 16; ++n) {
        const float2 u = *reinterpret_cast<const float2*>(b + r0 * C::kJoinPitch + 8 * n + cq);
        const float2 v = *reinterpret_cast<const float2*>(b + (r0 + 8) * C::kJoinPitch + 8 * n + cq);
        acc[n][0] += u.x; acc[n][1] += u.y; acc[n][2] += v.x; acc[n][3] += v.y;
      }
    };
    float* mybuf = join + (ks >> 1) * (16 * C::kJoinPitch);
    if (ks & 1) put(mybuf);
    if (!meet()) { ok = false; break; }
    if (!(ks & 1)) add(mybuf);
    if (ks == 2) put(mybuf);
    if (!meet()) { ok = false; break; }
    if (ks == 0) {
      add(join + 16 * C::kJoinPitch);
      const bool whole = p.c0 == p.c1;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (!has[k]) continue;
        if (whole && a.direct) {
          const float inv = tot[k] > 0.f ? 1.f / tot[k] : 0.f;
#pragma unroll
          for (int n = 0; n < 16; ++n)
            store2<FP16>(a.O, a.out_f32, orow[k] * kD + 8 * n + cq, acc[n][2 * k] * inv, acc[n][2 * k + 1] * inv);
          if (a.lse && (lane & 3) == 0) a.lse[orow[k]] = lse_of(top[k], tot[k]);
          continue;
        }
        const int sl = 2 * blockIdx.x + (p.first ? 1 : 0);
        const size_t at = whole ? orow[k] : (size_t)sl * a.part.rows + 16 * rt + r0 + 8 * k;
        float* dst = (whole ? a.part.dense[p.kind] : a.part.slots) + at * kD;
#pragma unroll
        for (int n = 0; n < 16; ++n)
          *reinterpret_cast<float2*>(dst + 8 * n + cq) = make_float2(acc[n][2 * k], acc[n][2 * k + 1]);
        if ((lane & 3) == 0) (whole ? a.part.dense_ml[p.kind] : a.part.slots_ml)[at] = make_float2(top[k], tot[k]);
      }
    }
  }
  if (!ok && lane == 0) set_error(kErrTimeout);
}

// ---------------------------------------------------------------------------
// The join: a warp per query row adds the row's parts (the prefix's, then the
// own keys', each in CTA order, so the result does not depend on timing).

struct JoinSide {
  PagedPart part;
  PagedCut c;
  const int64_t* units;
  int n;              // CTAs of the kernel that wrote it
  int on;
};

struct JoinArgs {
  PagedGeom g;
  JoinSide prefix, own;
  const int2* meta;
  void* O;
  float* lse;
  int out_f32;
};

struct RowSum {
  float m, l;
  float4 o;
};
__device__ __forceinline__ void row_add(RowSum& s, float2 ml, float4 o) {
  if (ml.x == -INFINITY && ml.y == 0.f) return;  // saw no key
  const float m = fmaxf(s.m, ml.x);
  const float f = ex2_approx(s.m - m), h = ex2_approx(ml.x - m);
  s.m = m;
  s.l = s.l * f + ml.y * h;
  s.o = make_float4(s.o.x * f + o.x * h, s.o.y * f + o.y * h, s.o.z * f + o.z * h, s.o.w * f + o.w * h);
}
__device__ __forceinline__ void side_add(RowSum& s, const JoinSide& d, int kind, size_t row, int tile_row, int c0,
                                         int c1, int stride, int offset, int lane) {
  if (c0 == c1) {
    row_add(s, d.part.dense_ml[kind][row], reinterpret_cast<const float4*>(d.part.dense[kind] + row * kD)[lane]);
    return;
  }
  const int64_t U = *d.units;
  const int n = d.n / stride;
#pragma unroll 4
  for (int c = c0; c <= c1; ++c) {
    if (share_begin(U, n, c) == share_begin(U, n, c + 1)) continue;  // a share without units
    const size_t at = (size_t)(2 * (c * stride + offset) + (c == c0 ? 1 : 0)) * d.part.rows + tile_row;
    row_add(s, d.part.slots_ml[at], reinterpret_cast<const float4*>(d.part.slots + at * kD)[lane]);
  }
}

template <bool FP16>
__global__ void __launch_bounds__(256) k_paged_join(const __grid_constant__ JoinArgs a) {
  const PagedGeom& g = a.g;
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int t = (int)(row / g.Hq), h = (int)(row % g.Hq);
  const int ntok = batch_tokens(g);
  if (t >= ntok) return;
  const int kvh = h / g.G, hh = h - kvh * g.G;
  RowSum s = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  int2 own = make_int2(0, 0);
  if (a.own.on) {
    own = a.meta[(int64_t)t * g.Hkv + kvh];
    own.x = max(0, min(own.x, a.own.n - 1));  // rows of a refused sequence were never written
    own.y = max(own.x, min(own.y, a.own.n - 1));
    if (!a.prefix.on && own.x == own.y) return;  // already the result
  }
  if (a.prefix.on) {
    const PagedCut& c = a.prefix.c;
    const int npt = (ntok + c.tpt - 1) / c.tpt, rt = t / c.tpt;
    const int64_t np = ((int64_t)g.prefix + (1 << c.kt_log2) - 1) >> c.kt_log2;
    const int team = team_size(c, npt, a.prefix.n), n = a.prefix.n / team;
    const int64_t u0 = (team > 1 ? (int64_t)kvh : (int64_t)kvh * npt + rt) * np, U = *a.prefix.units;
    side_add(s, a.prefix, 0, row, (t - rt * c.tpt) * g.G + hh, share_owner(U, n, u0), share_owner(U, n, u0 + np - 1),
             team, team > 1 ? rt : 0, lane);
  }
  if (a.own.on) {
    int tr = hh;
    if (own.x != own.y) {  // the token's place in its row tile
      const int q0 = g.q_start[seq_of_token(g.q_start, g.nseq, t)];
      tr = max(0, (t - q0) % a.own.c.tpt) * g.G + hh;
    }
    side_add(s, a.own, 1, row, tr, own.x, own.y, 1, 0, lane);
  }
  const float inv = s.l > 0.f ? 1.f / s.l : 0.f;
  if (a.out_f32)
    reinterpret_cast<float4*>(static_cast<float*>(a.O) + row * kD)[lane] =
        make_float4(s.o.x * inv, s.o.y * inv, s.o.z * inv, s.o.w * inv);
  else
    reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.O) + row * kD)[lane] =
        make_uint2(pack2<FP16>(s.o.x * inv, s.o.y * inv), pack2<FP16>(s.o.z * inv, s.o.w * inv));
  if (a.lse && lane == 0) a.lse[row] = lse_of(s.m, s.l);
}

}  // namespace s2o
