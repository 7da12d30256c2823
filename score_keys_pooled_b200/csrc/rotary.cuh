// Rotary positions with several axes, and the paged-cache append that applies
// them on the way.
//
// A head row x of a token is turned pair by pair: frequency f (of rot / 2)
// belongs to one position axis, its angle is phi = p[axis(f)] * inv_freq[f],
// and the pair (a, b) becomes (a cos phi - b sin phi, a sin phi + b cos phi).
// The pair of f is (x[f], x[f + rot/2]) ("half") or (x[2f], x[2f+1])
// ("adjacent"); elements from rot on pass through.  The inverse turns by -phi:
// the transposed rotation, which is also the gradient's way back.
//
// Angles: the host hands over inv_freq / 2 pi, so p * that is the angle in
// turns, formed in fp64; only its fraction (exact after the subtraction of the
// nearest integer) goes to fp32, so an angle is within 1e-6 rad at positions
// up to 2^31 and within 4e-7 below 2^28.  The products and the sum are fp32,
// rounded once to the type.
//
// Both kernels are bound by memory: a row of 256 bytes is read once and
// written once, 16 bytes a load, eight lanes a row (a lane owns eight pairs:
// two 16-byte chunks).  A block takes the rows of `tb` tokens; each token's
// angles are formed once per block and shared by all of its heads.  The
// rotation of 131072 tokens of 40 heads, 2.68 GB, takes 442 us, 6.1 TB/s or 93 %
// of the measured copy rate; the append of 14336 tokens, 353 MB whose cache rows
// lie 256 bytes here and there, 70 us, 5.1 TB/s; one row more or fewer in flight
// a thread and larger or smaller blocks made either slower or no faster.
#pragma once

#include <cuda_fp16.h>

#include "row_views.h"
#include "s2o_common.cuh"

namespace s2o {

constexpr int kRotThreads = 128;      // 256 threads and 8 tokens: 78 us where this takes 76.5 (2 x 9973 tokens, 40 heads)
constexpr int kRotMaxTokens = 4;      // tokens of a block
constexpr unsigned kErrBadCache = 8u;  // device error word: page id, length or token range out of range

struct RotaryTable {
  double turns[64];   // inv_freq / (2 pi)
  uint8_t axis[64];
  int rot, adjacent, naxes;
  float sign;         // -1: inverse
};

template <bool FP16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if (FP16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(bf16_lo(w), bf16_hi(w));
}
template <bool FP16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if (FP16) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  return pack_bf16x2(lo, hi);
}

// cos and sin of the tb tokens' angles into shared memory.  Lane j of a row
// reads its pairs 8j .. 8j+7 as four 16-byte words {c, s, c, s}; word k of
// lane j is at [k][j], so the eight lanes of a row read 128 consecutive bytes.
__device__ __forceinline__ void fill_angles(float4 (*cs)[4][8], const RotaryTable& r, int ntok,
                                            const int32_t (*pos)[3]) {
  const int F = r.rot >> 1;
  for (int i = threadIdx.x; i < ntok * 64; i += kRotThreads) {
    const int tok = i >> 6, f = i & 63;
    if (f >= F) continue;
    const double turns = (double)pos[tok][r.axis[f]] * r.turns[f];
    float s, c;
    sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
    float2* w = reinterpret_cast<float2*>(&cs[tok][(f & 7) >> 1][f >> 3]) + (f & 1);
    *w = make_float2(c, r.sign * s);
  }
}

// lane j of a row: both chunks of its eight pairs, turned; or copied
// (STREAM: read and written past the caches' use, which the append's scattered
// rows gain by, 72 -> 70 us for 14k tokens, and the rotation's lose by)
template <bool FP16, bool STREAM>
__device__ __forceinline__ void turn_row(const uint16_t* src, uint16_t* dst, int j, bool rotate, const RotaryTable& r,
                                         const float4 (*cs)[8]) {
  const bool turn = rotate && 16 * j < r.rot;
  // element offsets of the lane's two chunks
  const int e0 = turn && !r.adjacent ? 8 * j : 16 * j;
  const int e1 = turn && !r.adjacent ? 8 * j + (r.rot >> 1) : 16 * j + 8;
  const uint4* s0 = reinterpret_cast<const uint4*>(src + e0);
  const uint4* s1 = reinterpret_cast<const uint4*>(src + e1);
  uint4 a = STREAM ? __ldcs(s0) : *s0;
  uint4 b = STREAM ? __ldcs(s1) : *s1;
  if (turn) {
    uint32_t* aw = reinterpret_cast<uint32_t*>(&a);
    uint32_t* bw = reinterpret_cast<uint32_t*>(&b);
    if (!r.adjacent) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 t = cs[k][j];
        const float2 x = unpack2<FP16>(aw[k]), y = unpack2<FP16>(bw[k]);
        aw[k] = pack2<FP16>(x.x * t.x - y.x * t.y, x.y * t.z - y.y * t.w);
        bw[k] = pack2<FP16>(x.x * t.y + y.x * t.x, x.y * t.w + y.y * t.z);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {  // pairs 2k, 2k + 1 are words 2k, 2k + 1 of the 32 bytes
        const float4 t = cs[k][j];
        uint32_t& w0 = k < 2 ? aw[2 * k] : bw[2 * k - 4];
        uint32_t& w1 = k < 2 ? aw[2 * k + 1] : bw[2 * k - 3];
        const float2 x = unpack2<FP16>(w0), y = unpack2<FP16>(w1);
        w0 = pack2<FP16>(x.x * t.x - x.y * t.y, x.x * t.y + x.y * t.x);
        w1 = pack2<FP16>(y.x * t.z - y.y * t.w, y.x * t.w + y.y * t.z);
      }
    }
  }
  uint4* d0 = reinterpret_cast<uint4*>(dst + e0);
  uint4* d1 = reinterpret_cast<uint4*>(dst + e1);
  if (STREAM) {
    __stcs(d0, a);
    __stcs(d1, b);
  } else {
    *d0 = a;
    *d1 = b;
  }
}

struct RotaryArgs {
  RotaryTable r;
  RowView q, k, qo, ko;
  const int32_t* pos;  // [naxes, B, N]
  int B, N, Hq, Hkv, tb;
};

template <bool FP16>
__global__ void __launch_bounds__(kRotThreads) k_rotary(const __grid_constant__ RotaryArgs a) {
  __shared__ float4 cs[kRotMaxTokens][4][8];
  __shared__ int32_t pos[kRotMaxTokens][3];
  const int64_t total = (int64_t)a.B * a.N;
  const int64_t t0 = (int64_t)blockIdx.x * a.tb;
  const int ntok = (int)min((int64_t)a.tb, total - t0);
  if (threadIdx.x < ntok * 3) {
    const int tok = threadIdx.x / 3, ax = threadIdx.x % 3;
    if (ax < a.r.naxes) pos[tok][ax] = a.pos[ax * total + t0 + tok];
  }
  __syncthreads();
  fill_angles(cs, a.r, ntok, pos);
  __syncthreads();
  const int H = a.Hq + a.Hkv, j = threadIdx.x & 7;
  for (int i = threadIdx.x >> 3; i < ntok * H; i += kRotThreads / 8) {
    const int tok = i / H, h = i - tok * H;
    const int64_t bt = t0 + tok, b = bt / a.N, t = bt - b * a.N;
    const bool isq = h < a.Hq;
    const RowView& in = isq ? a.q : a.k;
    const RowView& out = isq ? a.qo : a.ko;
    const int hh = isq ? h : h - a.Hq;
    turn_row<FP16, false>(in.p + b * in.sb + t * in.st + hh * in.sh, out.p + b * out.sb + t * out.st + hh * out.sh, j, true,
                   a.r, cs[tok]);
  }
}

struct AppendArgs {
  RotaryTable r;
  RowView q, k, v, qo;       // q.p null: no queries; sb unused
  const int32_t* pos;        // [naxes, Tq] or null: prefix_len + place in the sequence, on every axis
  const int32_t* table;      // [nseq, max_pages]
  const int32_t* q_start;    // [nseq + 1]
  const int32_t* kv_len;     // [nseq]
  uint16_t *kc, *vc;         // [num_pages, Hkv, page, 128]
  int Hq, Hkv, page_log2, num_pages, nseq, max_pages, Tq, max_q, prefix, tb;
};

// A sequence's numbers, as a call may find them on the device: tokens [q0, q1)
// behind one another from 0 to at most Tq, at most max_q of them, `len` own keys
// that hold them and fit the table.  One without tokens needs no length, and its
// place is its neighbours' to answer for.
__device__ __forceinline__ bool seq_fits(int s, int q0, int q1, int len, int Tq, int max_q, int64_t room) {
  const int64_t n = (int64_t)q1 - q0;
  if (n == 0 && (s > 0 || q0 == 0)) return true;
  return !(q0 < 0 || (s == 0 && q0 != 0) || n < 0 || q1 > Tq || n > max_q || len < n || len > room);
}

// the sequence of token t: the last s with q_start[s] <= t (q_start[0] <= t)
__device__ __forceinline__ int seq_of_token(const int32_t* q_start, int nseq, int t) {
  int lo = 0, hi = nseq;  // q_start[lo] <= t; the answer is in [lo, hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (q_start[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

template <bool FP16>
__global__ void __launch_bounds__(kRotThreads) k_cache_append(const __grid_constant__ AppendArgs a) {
  __shared__ float4 cs[kRotMaxTokens][4][8];
  __shared__ int32_t pos[kRotMaxTokens][3];
  __shared__ int64_t slot[kRotMaxTokens];  // row of head 0 in the caches; -1: no write
  const int t0 = blockIdx.x * a.tb;
  const int64_t room = (int64_t)a.max_pages << a.page_log2;
  // The blocks check every sequence between them, those that none of the tokens
  // below leads to as well.  The first warp has the tokens; the others' reads
  // are on their way beside its own.
  if (threadIdx.x >= 32)
    for (int64_t s = (int64_t)blockIdx.x * (kRotThreads - 32) + threadIdx.x - 32; s < a.nseq;
         s += (int64_t)gridDim.x * (kRotThreads - 32))
      if (!seq_fits((int)s, a.q_start[s], a.q_start[s + 1], a.kv_len[s], a.Tq, a.max_q, room)) set_error(kErrBadCache);
  const int ntok = min(min(a.tb, a.Tq - t0), a.q_start[a.nseq] - t0);  // tokens behind the last sequence: none
  if (ntok <= 0) return;
  if (threadIdx.x < ntok) {
    const int t = t0 + threadIdx.x;
    const int s = seq_of_token(a.q_start, a.nseq, t);
    const int q0 = a.q_start[s], q1 = a.q_start[s + 1], len = a.kv_len[s];
    const int64_t at = (int64_t)len - q1 + t;  // place among the sequence's own keys
    bool ok = q0 <= t && t < q1 && seq_fits(s, q0, q1, len, a.Tq, a.max_q, room);
    int64_t row = -1;
    if (ok) {
      const int page = a.table[(int64_t)s * a.max_pages + (at >> a.page_log2)];
      if (page < 0 || page >= a.num_pages) ok = false;
      else row = (((int64_t)page * a.Hkv) << a.page_log2) + (at & ((1 << a.page_log2) - 1));
    }
    if (!ok) set_error(kErrBadCache);
    slot[threadIdx.x] = row;
#pragma unroll
    for (int ax = 0; ax < 3; ++ax)
      if (ax < a.r.naxes) pos[threadIdx.x][ax] = a.pos ? a.pos[(int64_t)ax * a.Tq + t] : (int32_t)(a.prefix + at);
  }
  __syncthreads();
  fill_angles(cs, a.r, ntok, pos);
  __syncthreads();
  const int Hq = a.q.p ? a.Hq : 0, H = Hq + 2 * a.Hkv, j = threadIdx.x & 7;
  for (int i = threadIdx.x >> 3; i < ntok * H; i += kRotThreads / 8) {
    const int tok = i / H, t = t0 + tok;
    int h = i - tok * H;
    if (h < Hq) {
      turn_row<FP16, true>(a.q.p + t * a.q.st + h * a.q.sh, a.qo.p + t * a.qo.st + h * a.qo.sh, j, true, a.r, cs[tok]);
      continue;
    }
    if (slot[tok] < 0) continue;
    h -= Hq;
    const bool isk = h < a.Hkv;
    if (!isk) h -= a.Hkv;
    const RowView& in = isk ? a.k : a.v;
    turn_row<FP16, true>(in.p + t * in.st + h * in.sh, (isk ? a.kc : a.vc) + (slot[tok] + ((int64_t)h << a.page_log2)) * kD, j,
                   isk, a.r, cs[tok]);
  }
}

}  // namespace s2o
