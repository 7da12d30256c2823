// Attention over a paged cache, many query rows a KV head: the shared prefix
// against the rows of the whole batch, or long chunks of new tokens against
// the prefix and their own keys.
//
// Bound by the tensor core and the exponentials: 256 rows against a key and
// its value are 4 d * 256 flops for 512 bytes, 256 flops a byte, where HBM
// stops being the limit.  An item's row tile is therefore 256 rows, two
// tcgen05 tiles of 128 (G query heads of 128 / G tokens each), that share
// every K/V tile; roles, tensor-memory layout, chunked softmax and register
// split are those of k_sparse_attn2 (see there), with these differences:
//   * S is double buffered, P written over the scores it came from (O and S fill
//     the 512 columns), so that the products of the next half tile run during
//     the softmax of this one: 256 sequences behind a 128K prefix, 598 us with
//     one buffer, 582 with two.  A half tile of both heads takes about 1840
//     clocks, of which the products are 1280 (64-key scores read Q again for
//     half the work, 48 clocks a step where 32 would do) and the exponentials
//     1024; one product of 128 keys (673 us: the heads fall into step and wait
//     together), one issuer for both heads (594 and 679) and turns at the
//     exponentials (596) were slower.  Repeated for long it is the power limit
//     that holds it: 526 us a pass over 20 passes, 609 over 3000;
//   * keys come from pages: warps 9 and 10 issue TMA boxes (64 columns x
//     min(page, 64) rows, 128-byte swizzle) into the K and V rings; the last
//     tile of a list that ends inside it has its missing V rows zeroed in
//     shared memory before the tensor core may read them (0 * NaN);
//   * Q tiles are TMA boxes of 64 columns x G heads x 128 / G tokens, fetched
//     by the head's issuer as soon as the softmax has taken the last scores of
//     the piece before;
//   * a CTA walks the pieces of its share (paged_sched.cuh): warp 9 announces
//     each in a small ring that every role follows, all barriers keep counting
//     across pieces, and the first P V of a piece waits until the softmax warps
//     have read the piece before it out of tensor memory;
//   * a piece that is not the whole answer leaves fp32 accumulators and
//     (reference, sum) for the join.
#pragma once
#include "paged_attn.cuh"
#include "sparse_attn2.cuh"

namespace s2o {

constexpr int kPtKeys = 128;  // keys of a tile
constexpr int kPieceSlots = 4;
constexpr uint32_t kPtOffBar = kOff2V + kStagesV * kTile2Bytes;
constexpr uint32_t kPtOffPiece = kPtOffBar + 48 * 8;
constexpr uint32_t kPtOffRed = kPtOffPiece + kPieceSlots * 64;
constexpr uint32_t kPtSmemData = kPtOffRed + 36 * 8;
constexpr size_t kPtSmem = kPtSmemData + 1024;
static_assert(kPtSmem <= 227 * 1024, "shared memory");

// barrier slots; those of k_sparse_attn2 up to the P and O ones
constexpr int kPtSFull = kBarSFull;  // [2][2] MMA commit (S_i,b written) -> softmax i; slot + 2 i + b
constexpr int kPtOFree = 23;       // [2] softmax i, one arrive per warp: O_i was read -> issuer i
constexpr int kPtVTmp = 25;        // V loader's own: boxes of a ragged tile landed
constexpr int kPtDrain = 26;       // [2]
constexpr int kPtQFull = 28;       // [2] Q tile i landed -> issuer i
constexpr int kPtPieceFull = 30;   // [kPieceSlots]
constexpr int kPtPieceEmpty = 34;  // [kPieceSlots] V loader, 2 issuers, 8 softmax warps
constexpr int kPtBars = 38;
constexpr int kPtSlotTmem = 40;

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// two score buffers of 64 keys a head; P (32 columns) takes the place of the
// scores it was made from
__device__ __forceinline__ uint32_t col_sp(int i, int b) { return 256u + 128u * i + 64u * b; }

// Shared-memory descriptors of 128-byte swizzled tiles as two words: the high
// one is the same for all (8-row groups 1024 bytes apart, version 1, swizzle),
// the low one holds address / 16, to which offsets / 16 are added, and the
// leading dimension's offset (see sdesc_sw128).
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo_bytes) {
  return ((saddr >> 4) & 0x3FFFu) | ((lbo_bytes >> 4) << 16);
}
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n"
      " setp.ne.b32 p, %4, 0;\n mov.b64 a, {%1, %5};\n mov.b64 b, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(add), "r"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 b;\n"
      " setp.ne.b32 p, %4, 0;\n mov.b64 b, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(add), "r"(kDescHi)
      : "memory");
}

// tile t of a piece: its page list, first key in it, and the keys the piece's
// rows can reach there
struct TileKeys {
  const int32_t* list;
  int key0, valid;
};
__device__ __forceinline__ TileKeys tile_keys(const PagedGeom& g, const Piece& p, int t) {
  TileKeys k;
  if (p.kind == 0 || t < p.np) {
    k.list = g.prefix_pages;
    k.key0 = t * kPtKeys;
    k.valid = min(kPtKeys, g.prefix - k.key0);
  } else {
    k.list = g.table + (int64_t)p.seq * g.max_pages;
    k.key0 = (t - p.np) * kPtKeys;
    k.valid = min(kPtKeys, p.len - k.key0);
  }
  return k;
}

// 16 rows (of tensor-memory lanes) of 32 columns, as matrix fragments: thread
// 4 i + q has columns 8 j + 2 q + {0, 1} of row i in v[4 j], v[4 j + 1], of row
// i + 8 in v[4 j + 2], v[4 j + 3]
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, float* v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

template <bool FP16>
__global__ void __launch_bounds__(kAttn2Threads, 1)
    k_paged_tile(const __grid_constant__ PagedArgs a, const __grid_constant__ CUtensorMap tmQ,
                 const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* sgen = smem_raw + (sbase - smem_u32(smem_raw));
  auto bar = [&](int k) { return sbase + kPtOffBar + 8u * (uint32_t)k; };
  auto piece_at = [&](int k) { return reinterpret_cast<Piece*>(sgen + kPtOffPiece + 64 * k); };
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(sgen + kPtOffBar + 8 * kPtSlotTmem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const PagedGeom& g = a.g;
  const int tpt = kLq / g.G;      // tokens of a 128-row tile
  const int trows = tpt * g.G;    // its rows

  let_next_start();
  if (tid == 0) {
    prefetch_map(&tmQ);
    prefetch_map(&tmK);
    prefetch_map(&tmV);
  }
  // side by side with the decode kernel: its items decide how many SMs are left
  SchedFound* found = reinterpret_cast<SchedFound*>(sgen + kPtOffRed + 34 * 8);
  const OwnRun run = own_run(g, a.beside ? a.other : a.c, 1, reinterpret_cast<int64_t*>(sgen + kPtOffRed), found);
  const int ctas =
      gridDim.x - (a.beside ? decode_sms(g, a.c, batch_tokens(g), run.total, a.own_ns, gridDim.x) : 0);
  if (blockIdx.x >= ctas) return;  // an SM for the decode kernel
  if (tid < kPtBars) {
    uint32_t count = 1;
    if ((tid >= kBarPFull && tid < kBarPFull + 4) || (tid >= kPtOFree && tid < kPtOFree + 2)) count = 4;
    if ((tid >= kBarKEmpty && tid < kBarKEmpty + kStagesK) || (tid >= kBarVEmpty && tid < kBarVEmpty + kStagesV)) count = 2;
    if (tid >= kPtPieceEmpty) count = 11;
    mbar_init(bar(tid), count);
    fence_mbar_init();
  }
  // Q rows that no box fills (128 is no multiple of G): zero
  for (int i = tid; i < (kLq - trows) * 2 * 16; i += kAttn2Threads) {
    const int row = trows + (i >> 5), qi = (i >> 4) & 1, ch = i & 15;
    *reinterpret_cast<uint4*>(sgen + kOff2Q + qi * kTile2Bytes + (ch >> 3) * (128 * 128) + swz128(row, ch & 7)) =
        make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32((const void*)tmem_slot), kTmem2Cols);
    tmem_relinquish();
  }
  Sched sc = sched_begin(g, a.c, 1, 0, ctas, run, found);
  if (tid == 0 && blockIdx.x == 0) *a.head = {sc.U, ctas};
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // the next piece, for every role but the one that announces them; done: kind < 0
  auto take_piece = [&](int pi, Piece& p) {
    const int slot = pi % kPieceSlots;
    if (!mbar_wait_bounded(bar(kPtPieceFull + slot), (pi / kPieceSlots) & 1)) return false;
    p = *piece_at(slot);
    return true;
  };
  auto rows_of = [&](const Piece& p, int i) { return max(0, min(tpt, p.ntok - i * tpt)) * g.G; };

  if (warp == kLoadWarp0 || warp == kLoadWarp0 + 1) {
    // ------------------------------------------------------------------ loaders
    regs_decrease<kRegsOther>();
    const bool is_k = warp == kLoadWarp0;
    const int nst = is_k ? kStagesK : kStagesV;
    const int bar_full = is_k ? kBarKFull : kBarVFull, bar_empty = is_k ? kBarKEmpty : kBarVEmpty;
    const uint32_t ring = sbase + (is_k ? kOff2K : kOff2V);
    const CUtensorMap* tm = is_k ? &tmK : &tmV;
    const int box_log2 = min(g.page_log2, 6), rest_log2 = g.page_log2 - box_log2;
    const int bi = lane >> 1, half = lane & 1;  // this lane's box of a tile
    bool ok = true;
    uint32_t it = 0, vt = 0;
    // own chunks are read by tile after tile, and the prefix by all of them
    const uint64_t policy = keys_policy(!a.c.own_items && (sc.npt <= 1 || sc.team > 1));
    SplitItem split = {0, 0, 0, 0};
    for (int pi = 0; ok; ++pi) {
      Piece p;
      if (is_k) {
        p = sched_next(g, a.c, sc);
        const int slot = pi % kPieceSlots;
        if (!warp_ok(mbar_wait_bounded(bar(kPtPieceEmpty + slot), ((pi / kPieceSlots) & 1) ^ 1))) { ok = false; break; }
        if (lane == 0) {
          *piece_at(slot) = p;
          mbar_arrive(bar(kPtPieceFull + slot));
        }
        announce_split(a, sc, p, split, lane);
        if (p.kind < 0) break;
      } else {
        if (!warp_ok(take_piece(pi, p))) { ok = false; break; }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kPtPieceEmpty + pi % kPieceSlots));
        if (p.kind < 0) break;
      }
      // page of this lane's box, one tile ahead
      auto page_of = [&](int t) {
        if (t >= p.tile1) return 0;
        const TileKeys k = tile_keys(g, p, t);
        if ((bi << box_log2) >= k.valid) return 0;
        return checked_page(g, k.list, ((k.key0 >> box_log2) + bi) >> rest_log2);
      };
      int page_next = page_of(p.tile0);
      for (int t = p.tile0; t < p.tile1; ++t, ++it) {
        const int page = page_next;
        page_next = page_of(t + 1);
        const TileKeys k = tile_keys(g, p, t);
        const int nb = (k.valid + (1 << box_log2) - 1) >> box_log2;
        const int st = it % nst;
        if (!warp_ok(mbar_wait_bounded(bar(bar_empty + st), ((it / nst) & 1) ^ 1))) { ok = false; break; }
        const bool ragged = !is_k && k.valid < kPtKeys;
        const uint32_t full = bar(ragged ? kPtVTmp : bar_full + st);
        if (lane == 0) mbar_expect_tx(full, (uint32_t)nb << (box_log2 + 8));
        __syncwarp();
        if (bi < nb) {
          const int in_page = (((k.key0 >> box_log2) + bi) & ((1 << rest_log2) - 1)) << box_log2;
          tma_load_rows(ring + st * kTile2Bytes + half * (128 * 128) + (bi << box_log2) * 128, tm, 64 * half,
                        ((page * g.Hkv + p.kvh) << g.page_log2) + in_page, full, policy);
        }
        if (ragged) {
          const bool landed = warp_ok(mbar_wait_bounded(full, vt & 1));
          ++vt;
          if (!landed) { ok = false; ++it; break; }
          for (int i = lane; i < (kPtKeys - k.valid) * 16; i += 32) {
            const int row = k.valid + (i >> 4), ch = i & 15;
            *reinterpret_cast<uint4*>(sgen + (ring - sbase) + st * kTile2Bytes + (ch >> 3) * (128 * 128) +
                                      swz128(row, ch & 7)) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(bar_full + st));
        }
      }
    }
    if (!ok && lane == 0) {
      set_error(kErrTimeout);
      if (a.split && is_k) a.split[blockIdx.x] = {0, 0, 0, 0};
    }
    // nothing may land in shared memory after the CTA ends
    for (uint32_t k = it > (uint32_t)nst ? it - nst : 0; k < it; ++k)
      if (!mbar_wait_bounded(bar(bar_full + k % nst), (k / nst) & 1)) {
        if (lane == 0) set_error(kErrTimeout);
      }
  } else if (warp == kMmaWarp || warp == kMmaWarp1) {
    // ------------------------------------------------------------------ MMA issuers
    regs_decrease<kRegsOther>();
    const int i = warp == kMmaWarp ? 0 : 1;
    if (lane == 0) {
      constexpr uint32_t kTypes = FP16 ? 0u : (1u << 7) | (1u << 10);
      const uint32_t idesc_qk = (idesc_bf16_f32(128, kBk, false) & ~((7u << 7) | (7u << 10))) | kTypes;
      const uint32_t idesc_pv = (idesc_bf16_f32(128, 128, true) & ~((7u << 7) | (7u << 10))) | kTypes;
      bool ok = true;
      uint32_t ks = 0, kph = 0, vs = 0, vph = 0;  // ring stages and their parities
      uint32_t gt = 0;  // tiles of this head so far
      uint32_t np = 0;  // pieces this head had rows in
      uint32_t nq = 0;  // Q tiles asked for
      const uint32_t tS = tmem + col_sp(i, 0), tO = tmem + col_o(i);
      const uint32_t lo_q = desc_lo(sbase + kOff2Q + i * kTile2Bytes, 16);
      const uint32_t lo_k = desc_lo(sbase + kOff2K, 16), lo_v = desc_lo(sbase + kOff2V, 128 * 128);
      auto wait = [&](int slot, uint32_t parity) {
        ok = ok && mbar_wait_bounded(bar(slot), parity);
        return ok;
      };
      auto fetch_q = [&](const Piece& p) {
        if (p.kind < 0 || rows_of(p, i) == 0) return;
        mbar_expect_tx(bar(kPtQFull + i), (uint32_t)trows * 256);
        for (int h = 0; h < 2; ++h)
          tma_load_3d(sbase + kOff2Q + i * kTile2Bytes + h * (128 * 128), &tmQ, 64 * h, p.kvh * g.G, p.tok0 + i * tpt,
                      bar(kPtQFull + i));
        ++nq;
      };
      // S of half h of the K stage: 8 products of 16 columns.  What the softmax
      // left in that buffer, P, was read by a product issued before
      auto qk = [&](int h) {
        tc_fence_after();
        const uint32_t k0 = lo_k + ks * (kTile2Bytes >> 4) + h * (kBk * 128 >> 4);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t at = (kk >> 2) * (128 * 128 >> 4) + (kk & 3) * 2;
          mma_ss(tS + kBk * h, lo_q + at, k0 + at, idesc_qk, kk > 0 ? 1u : 0u);
        }
        tc_commit(bar(kPtSFull + 2 * i + h));
        if (h == 1) {
          tc_commit(bar(kBarKEmpty + ks));
          if (++ks == kStagesK) { ks = 0; kph ^= 1; }
        }
      };
      // O (+)= P of half h times that half of the V stage: 4 products of 16 keys
      auto pv = [&](int h, bool add) {
        tc_fence_after();
        const uint32_t v0 = lo_v + vs * (kTile2Bytes >> 4) + h * (kBk * 128 >> 4);
#pragma unroll
        for (int kk = 0; kk < kBk / 16; ++kk)
          mma_ts(tO, tS + kBk * h + 8 * kk, v0 + kk * (16 * 128 >> 4), idesc_pv, add || kk > 0 ? 1u : 0u);
        tc_commit(bar(kBarODone + 2 * i + h));
        if (h == 1) {
          tc_commit(bar(kBarVEmpty + vs));
          if (++vs == kStagesV) { vs = 0; vph ^= 1; }
        }
      };
      Piece p, next;
      ok = take_piece(0, next);
      if (ok) fetch_q(next);
      for (int pi = 0; ok; ++pi) {
        p = next;
        mbar_arrive(bar(kPtPieceEmpty + pi % kPieceSlots));
        if (p.kind < 0) break;
        const int ntiles = p.tile1 - p.tile0;
        if (rows_of(p, i) == 0) {  // let the stages pass
          for (int t = 0; ok && t < ntiles; ++t) {
            if (!wait(kBarKFull + ks, kph)) break;
            mbar_arrive(bar(kBarKEmpty + ks));
            if (++ks == kStagesK) { ks = 0; kph ^= 1; }
            if (!wait(kBarVFull + vs, vph)) break;
            mbar_arrive(bar(kBarVEmpty + vs));
            if (++vs == kStagesV) { vs = 0; vph ^= 1; }
          }
          if (ok) ok = take_piece(pi + 1, next);
          if (ok) fetch_q(next);
          continue;
        }
        // half a tile at a time, two S buffers: P V of a half, then S of the same
        // half of the next tile into its buffer, so the softmax finds its next
        // scores ready.  The thread does little but issue: descriptors are a
        // base plus constants, stages and parities are counted, since its
        // instructions, one warp's chain, are what the tensor core waits for.
        if (!wait(kPtQFull + i, np & 1) || !wait(kBarKFull + ks, kph)) break;
        qk(0);
        qk(1);
        for (int t = 0; t < ntiles; ++t, ++gt) {
          const bool more = t + 1 < ntiles;
          if (!wait(kBarVFull + vs, vph) || !wait(kBarPFull + 2 * i, gt & 1)) break;
          // the accumulator of the piece before this one has been read
          if (t == 0 && np > 0 && !wait(kPtOFree + i, (np - 1) & 1)) break;
          pv(0, t > 0);
          if (more) {
            if (!wait(kBarKFull + ks, kph)) break;
            qk(0);
          }
          if (!wait(kBarPFull + 2 * i + 1, gt & 1)) break;
          if (!more) {  // the softmax took the last scores: Q is free for the next piece
            ok = take_piece(pi + 1, next);
            if (!ok) break;
            fetch_q(next);
          }
          pv(1, true);
          if (more) qk(1);
        }
        if (!ok) break;
        ++np;
      }
      if (!ok) set_error(kErrTimeout);
      if (nq > 0 && !mbar_wait_bounded(bar(kPtQFull + i), (nq - 1) & 1)) set_error(kErrTimeout);
      tc_commit(bar(kPtDrain + i));
      if (!mbar_wait_bounded(bar(kPtDrain + i), 0)) set_error(kErrTimeout);
    }
  } else {
    // ------------------------------------------------------------------ softmax
    regs_increase<kRegsSoftmax>();
    constexpr float kShift = FP16 ? 7.f : 0.f;
    const int qi = warp >> 2;
    const int r = tid & 127;
    const int rt = r / g.G, rh = r - rt * g.G;  // token of the tile, head of the group
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tO = tmem + col_o(qi) + lane_base;
    bool ok = true;
    uint32_t gc = 0;
    for (int pi = 0; ok; ++pi) {
      Piece p;
      if (!warp_ok(take_piece(pi, p))) { ok = false; break; }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kPtPieceEmpty + pi % kPieceSlots));
      if (p.kind < 0) break;
      const int rows = rows_of(p, qi);
      if (rows == 0) continue;
      const bool has = r < rows;
      // keys the row sees: of the prefix all, of its own up to itself.  Rows of
      // nobody see what the last row sees: were they masked, their warp would
      // go through both forms of the exponentials below (one such warp in a CTA
      // made its tiles 20 % slower); a warp of them alone does nothing
      const int see_own = p.off + qi * tpt + min(rt, rows / g.G - 1) + 1;
      const int see_pre = g.prefix;
      const bool idle = (tid & 96) >= rows;
      float m_run = -INFINITY, ell = 0.f;
      const int nch = 2 * (p.tile1 - p.tile0);
      for (int c = 0; ok && c < nch; ++c) {
        const uint32_t n = gc + c;
        const int t = p.tile0 + (c >> 1);
        const bool pre = p.kind == 0 || t < p.np;
        const int vis = (pre ? see_pre - t * kPtKeys : see_own - (t - p.np) * kPtKeys) - kBk * (c & 1);
        const uint32_t tS = tmem + col_sp(qi, c & 1) + lane_base;
        if (!warp_wait(bar(kPtSFull + 2 * qi + (c & 1)), (n >> 1) & 1, kSpinLimit)) { ok = false; break; }
        tc_fence_after();
        if (idle) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBarPFull + 2 * qi + (c & 1)));
          continue;
        }
        // (one copy each of the long unrolled parts: the code is fetched anew in
        // every launch, through an L2 that the keys have passed through)
        // the first keys a row sees set its reference; a chunk whose sum passes
        // the limit moves it, and is done again from its scores
        float x[kBk], rs = 0.f;  // scores, then P as pairs; its sum
        bool set = __any_sync(0xffffffffu, m_run == -INFINITY);
        for (int pass = 0; pass < 2; ++pass) {
          tmem_ld32(tS, x);
          tmem_ld32(tS + 32, x + 32);
          tc_wait_ld();
          if (vis < kBk) {
#pragma unroll
            for (int k = 0; k < kBk; ++k)
              if (k >= vis) x[k] = -INFINITY;
          }
          if (set) {
            const bool move = m_run == -INFINITY || rs > kPgMove;
            float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int k = 0; k < kBk; k += 2) m4[(k >> 1) & 3] = fmax3(m4[(k >> 1) & 3], x[k], x[k + 1]);
            const float mt = fmaf(fmaxf(fmax3(m4[0], m4[1], m4[2]), m4[3]), kPgScale, -kShift);
            const float alpha = move && m_run != -INFINITY ? ex2_approx(m_run - mt) : 1.f;
            if (move) m_run = mt;
            ell *= alpha;
            if (c > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
              if (!warp_wait(bar(kBarODone + 2 * qi + ((n - 1) & 1)), ((n - 1) >> 1) & 1, kSpinLimit)) {
                ok = false;
                break;
              }
              tc_fence_after();
#pragma unroll 1
              for (int cc = 0; cc < 128; cc += 32) {
                float o[32];
                tmem_ld32(tO + cc, o);
                tc_wait_ld();
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] *= alpha;
                tmem_st32(tO + cc, o);
              }
            }
          }
          const float m = m_run == -INFINITY ? 0.f : m_run;
          const uint64_t s2 = f2_pack(kPgScale, kPgScale), nm2 = f2_pack(-m, -m);
          uint64_t rs2 = 0;
#pragma unroll
          for (int k = 0; k < kBk; k += 2) {
            const uint64_t v = f2_fma(f2_pack(x[k], x[k + 1]), s2, nm2);
            const float p0 = ex2_approx(f2_lo(v)), p1 = ex2_approx(f2_hi(v));
            rs2 = f2_add(rs2, f2_pack(p0, p1));
            x[k / 2] = __uint_as_float(pack2<FP16>(p0, p1));
          }
          rs = f2_lo(rs2) + f2_hi(rs2);
          set = __any_sync(0xffffffffu, rs > kPgMove);
          if (!set) break;
        }
        if (!ok) break;
        ell += rs;
        tmem_st32(tS, x);
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarPFull + 2 * qi + (c & 1)));
      }
      if (ok) {
        const uint32_t n = gc + nch - 1;
        ok = warp_wait(bar(kBarODone + 2 * qi + (n & 1)), (n >> 1) & 1, kSpinLimit);
      }
      if (!ok) break;
      gc += nch;
      tc_fence_after();
      const bool whole = p.first && p.last, final = whole && a.direct;
      const float inv = ell == 0.f ? 0.f : 1.f / ell;
      const size_t orow = (size_t)(p.tok0 + qi * tpt + rt) * g.Hq + p.kvh * g.G + rh;
      const int sl = 2 * p.share + (p.first ? 1 : 0);
      const size_t at = whole ? orow : (size_t)sl * a.part.rows + qi * trows + r;
      float* part = (whole ? a.part.dense[p.kind] : a.part.slots) + at * kD;
      if (!final) {
        // four threads a row, so that a store writes whole lines of eight rows: 256
        // sequences of short keys behind an 8K prefix 87.6 -> 85.6 us a pass against
        // a thread that writes its own row
        float* at_row[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          at_row[i] = reinterpret_cast<float*>(
              __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(has ? part : nullptr), 8 * i + lane / 4));
#pragma unroll 1
        for (int cc = 0; cc < 128; cc += 32) {
          float o[32];
          tmem_ld_frag(tO + cc, o);
          tmem_ld_frag(tO + (16u << 16) + cc, o + 16);
          tc_wait_ld();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float* v = o + 16 * (i >> 1) + 2 * (i & 1);
            if (at_row[i])
              store_part(at_row[i] + cc, lane & 3, v[0], v[1], v[4], v[5], v[8], v[9], v[12], v[13]);
          }
        }
      } else {
#pragma unroll 1
        for (int cc = 0; cc < 128; cc += 32) {
          float o[32];
          tmem_ld32(tO + cc, o);
          tc_wait_ld();
          if (!has) {
          } else if (a.out_f32) {
            float4* dst = reinterpret_cast<float4*>(static_cast<float*>(a.O) + orow * kD + cc);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              dst[k] = make_float4(o[4 * k] * inv, o[4 * k + 1] * inv, o[4 * k + 2] * inv, o[4 * k + 3] * inv);
          } else {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.O) + orow * kD + cc);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              dst[k] = make_uint4(pack2<FP16>(o[8 * k] * inv, o[8 * k + 1] * inv),
                                  pack2<FP16>(o[8 * k + 2] * inv, o[8 * k + 3] * inv),
                                  pack2<FP16>(o[8 * k + 4] * inv, o[8 * k + 5] * inv),
                                  pack2<FP16>(o[8 * k + 6] * inv, o[8 * k + 7] * inv));
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kPtOFree + qi));
      if (has) {
        if (!final) (whole ? a.part.dense_ml[p.kind] : a.part.slots_ml)[at] = make_float2(m_run, ell);
        else if (a.lse) a.lse[orow] = lse_of(m_run, ell);
      }
    }
    if (!ok && lane == 0) set_error(kErrTimeout);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmem2Cols);
  }
}

}  // namespace s2o
