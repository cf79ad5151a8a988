// A whole mixture-of-experts FFN for a few tokens: per-token E4M3
// quantization, expert up projection (optionally gated), activation, per-row
// E4M3 quantization of the hidden rows, expert down projection, weighted sum
// over a token's experts and residual.
//
//   a row is one (token, choice) pair, slot t * topk + j, with expert e:
//     z = (x_q . W_up[e]^T) * s_x * s_up[e]            fp32 sums of E4M3 products
//     h = fp16(act(z))  or, gated,  fp16(act(z[:F]) * z[F:])
//     y = (h_q . W_down[e]^T) * s_h * s_down[e]
//   out[t] = fp16(sum_j weight[t, j] * y[t, j] + residual[t])   fp32, j ascending
// x_q, s_x and h_q, s_h are the per-row codes and scales of quant_rows.cuh; the
// hidden rows are rounded to fp16 between the projections as on the grouped
// path, so both paths quantize the same values.
//
// Bound: with few tokens an expert sees a handful of rows, so the time is that of
// streaming the chosen experts' weights once from HBM.  The products run on
// mma.sync m16n8k32 (E4M3 x E4M3, fp32 accumulators; measured 1.1 cycles per
// instruction and SM on B200, where the weights arrive at 23 bytes a cycle and SM,
// one instruction per 22 cycles and 8 rows): 16 weight rows are the M operand and up
// to 8 rows an n-tile.  A tcgen05 tile would need 128 weight rows and its
// single-thread issue takes 26-42 ns per 32 bytes of K whatever the row count,
// 1.7 us and more for K = 2048 on the one chain, where here eight warps share K.
//
// Work: the chosen experts, each cut into segments of at most rmax rows; a segment
// is a run of blocks of 16 outputs.  Every CTA takes an equal share of
// the blocks of all segments.  For a segment it first quantizes the rows into
// shared memory; its warps then take blocks, S of them sharing a block's K
// (S by cost, per CTA).  A lane copies the 16-byte pieces of weight rows that its
// own MMA fragments need with cp.async into a private ring, kDepth pieces of 16
// rows x 128 bytes ahead across block and segment boundaries, so the
// copies need no barrier.  K may be permuted in a product as long as both
// operands agree: lane (g, t) holds bytes 16 t .. 16 t + 15 of a 64-byte group of
// row g, which is one 16-byte load per row for two MMAs, for both operands.
// The S partial sums of a block meet in shared memory and are added in fixed order.
#pragma once

#include "activation.cuh"
#include "quant_rows.cuh"

namespace fp8q {

constexpr int kMfThreads = 256;
constexpr int kMfWarps = kMfThreads / 32;
constexpr int kMfMaxRows = 1024;       // T * topk
constexpr int kMfMaxTopk = 8;
constexpr int kMfMaxExperts = 1024;
constexpr int kMfChunk = 128;          // K bytes of a ring piece
constexpr int kMfPieceBytes = 16 * kMfChunk;
constexpr int kMfMaxSmem = 232448;     // 227 KB

struct MoeFewParams {
  const __half* x;          // up: [T, K]; down: hidden [T * topk, K]
  const int32_t* experts;   // [T * topk], -1: none
  const uint8_t* w;         // [E, wrows, K] E4M3
  const float* s_w;         // [E, wrows]
  int rows;                 // T * topk
  int topk;
  int E;
  int K;
  int n_out;                // outputs of a row: F (up) or N (down)
  int act;                  // up: Activation
  __half* hidden;           // up: [T * topk, F]
  float* y;                 // down: [T * topk, N]
  int rmax;                 // rows of a segment, a multiple of 8
};

// Shared-memory layout, the same on host and device.
struct MoeFewLayout {
  int pitch;      // bytes of a row of codes; 64 mod 128 keeps even and odd rows on different banks
  int ring;       // offsets
  int part;
  int rows;
  int segs;
  int counts;
  int scales;
  int total;
};
__host__ __device__ constexpr int mf_part_units(int nt) { return nt >= 4 ? 8 : 2 * nt; }   // x 4 KB
__host__ __device__ inline MoeFewLayout mf_layout(int nt, int depth, int K, int rmax, int R, int E) {
  MoeFewLayout l;
  l.pitch = (K + kMfChunk - 1) / kMfChunk * kMfChunk + 64;
  l.ring = 0;
  l.part = kMfWarps * depth * kMfPieceBytes;
  l.scales = l.part + mf_part_units(nt) * kMfWarps * 512;
  l.rows = l.scales + 64 * 4;
  l.segs = l.rows + R * 4;
  l.counts = l.segs + R * 4;
  l.total = (l.counts + (E + 4) * 4 + 15) & ~15;   // then the codes: rmax * pitch
  return l;
}

__device__ __forceinline__ void mma_e4m3_m16n8k32(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                  uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One segment: expert (10 bits) | rows - 1 (6) | first entry in the row list (10).
__device__ __forceinline__ int mf_seg(int e, int cnt, int row0) { return e | (cnt - 1) << 10 | row0 << 16; }
__device__ __forceinline__ int mf_seg_expert(int s) { return s & 1023; }
__device__ __forceinline__ int mf_seg_count(int s) { return ((s >> 10) & 63) + 1; }
__device__ __forceinline__ int mf_seg_row0(int s) { return s >> 16; }

// Group the rows by expert: segs[] and the row list (slots by expert, ascending
// within one: the CTAs that share an expert cut it into the same segments).
// ex: [rows] ints of scratch.  Returns the number of segments.
__device__ __forceinline__ int mf_schedule(const MoeFewParams& p, int* rows, int* segs, int* counts, int* ex,
                                           bool report) {
  for (int e = threadIdx.x; e < p.E; e += kMfThreads) counts[e] = 0;
  __syncthreads();
  for (int r = threadIdx.x; r < p.rows; r += kMfThreads) {
    int e = __ldg(p.experts + r);
    if (e >= 0 && e < p.E) {
      atomicAdd(&counts[e], 1);   // integers: the order does not matter
    } else {
      if (e != -1 && report) raise_error(0x8u);
      e = -1;
    }
    ex[r] = e;
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    const int per = (p.E + 31) / 32;
    const int e0 = min(p.E, lane * per), e1 = min(p.E, e0 + per);
    int nr = 0, ns = 0;
    for (int e = e0; e < e1; ++e) {
      nr += counts[e];
      ns += (counts[e] + p.rmax - 1) / p.rmax;
    }
    int ar = nr, as = ns;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int vr = __shfl_up_sync(0xffffffffu, ar, o), vs = __shfl_up_sync(0xffffffffu, as, o);
      if (lane >= o) {
        ar += vr;
        as += vs;
      }
    }
    int r0 = ar - nr, s0 = as - ns;
    for (int e = e0; e < e1; ++e) {
      const int c = counts[e];
      counts[e] = r0;   // from here on: the expert's next entry in the row list
      for (int k = 0; k < c; k += p.rmax) segs[s0++] = mf_seg(e, min(p.rmax, c - k), r0 + k);
      r0 += c;
    }
    if (lane == 31) counts[p.E] = as;
    __syncwarp();
    for (int r0 = 0; r0 < p.rows; r0 += 32) {   // 32 rows at a time, in order
      const int r = r0 + lane;
      const int e = r < p.rows ? ex[r] : -1;
      const uint32_t same = __match_any_sync(0xffffffffu, e);
      const int rank = __popc(same & ((1u << lane) - 1u));
      const int at = e >= 0 ? counts[e] : 0;
      __syncwarp();
      if (e >= 0) {
        rows[at + rank] = r;
        if (rank == 0) counts[e] = at + __popc(same);
      }
      __syncwarp();
    }
  }
  __syncthreads();
  return counts[p.E];
}

// Quantize the rows of a segment into shared memory (codes [cnt][pitch], zero
// behind K up to the pitch's last chunk; scales).  One warp per row.
template <bool kUp>
__device__ __forceinline__ void mf_build_rows(const MoeFewParams& p, int seg, const int* rows, uint8_t* codes,
                                              int pitch, float* scales, int warp, int lane) {
  const int cnt = mf_seg_count(seg), row0 = mf_seg_row0(seg);
  const int nvec = p.K >> 3;
  const int nvec_pad = (p.K + kMfChunk - 1) / kMfChunk * (kMfChunk / 8);
  for (int i = warp; i < cnt; i += kMfWarps) {
    const int slot = rows[row0 + i];
    const uint4* src = reinterpret_cast<const uint4*>(p.x + static_cast<int64_t>(kUp ? slot / p.topk : slot) * p.K);
    float m = 0.0f;
    for (int j = lane; j < nvec; j += 32) m = absmax8(src[j], m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const RowScale rs = row_scale_from_amax(m);
    uint2* dst = reinterpret_cast<uint2*>(codes + i * pitch);
    for (int j = lane; j < nvec_pad; j += 32) dst[j] = j < nvec ? encode8(src[j], rs.r) : make_uint2(0u, 0u);
    if (lane == 0) scales[i] = rs.s;
  }
}

// Where a warp stands in its CTA's share: segment, first block of the round, chunk.
struct MfIter {
  int seg;
  int end;    // last block of the segment in this share, exclusive
  int base;   // first block of the round
  int c;      // next chunk of K
};

// NT: n-tiles of 8 rows a segment may have; kDepth: ring pieces per warp.
template <int NT, int kDepth, bool kUp, bool kGated>
__global__ void __launch_bounds__(kMfThreads) moe_few_kernel(const MoeFewParams p) {
  extern __shared__ __align__(128) uint8_t mf_smem[];
  constexpr int kTiles = kUp && kGated ? 2 : 1;   // 16-row weight tiles of a block of 16 outputs
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t4 = lane & 3;
  const MoeFewLayout L = mf_layout(NT, kDepth, p.K, p.rmax, p.rows, p.E);
  uint8_t* ring = mf_smem + L.ring + warp * kDepth * kMfPieceBytes;
  float* part = reinterpret_cast<float*>(mf_smem + L.part);
  float* scales = reinterpret_cast<float*>(mf_smem + L.scales);
  int* rows = reinterpret_cast<int*>(mf_smem + L.rows);
  int* segs = reinterpret_cast<int*>(mf_smem + L.segs);
  int* counts = reinterpret_cast<int*>(mf_smem + L.counts);
  uint8_t* codes = mf_smem + L.total;

  // The experts may come from the kernel just before the up projection.  The
  // down projection starts once every CTA of the up projection has passed this
  // wait, so the experts are there and only the hidden rows are waited for.
  if (kUp) {
    pdl_wait_prior_grid();
    pdl_launch_dependents();
  }
  const int nseg = mf_schedule(p, rows, segs, counts, reinterpret_cast<int*>(part), kUp && blockIdx.x == 0);
  const int nb = (p.n_out + 15) / 16;
  const int total = nseg * nb;
  const int lo = static_cast<int>(static_cast<int64_t>(total) * blockIdx.x / gridDim.x);
  const int hi = static_cast<int>(static_cast<int64_t>(total) * (blockIdx.x + 1) / gridDim.x);

  // S warps share a block's K: the cheapest in chunks a warp walks through.
  const int nc = (p.K + kMfChunk - 1) / kMfChunk;
  int S = 1, cost = 1 << 30;
#pragma unroll
  for (int s = 1; s <= kMfWarps / kTiles; s *= 2) {
    const int per_round = kMfWarps / (s * kTiles);
    const int c = ((hi - lo + per_round - 1) / per_round) * ((nc + s - 1) / s);
    if (s <= nc && c < cost) {
      cost = c;
      S = s;
    }
  }
  const int per_round = kMfWarps / (S * kTiles);   // blocks of a round
  const int ks = warp % S, tl = warp / S;
  const int my_block = tl / kTiles, sub = tl % kTiles;
  const int c0 = ks * nc / S, c1 = (ks + 1) * nc / S;
  const int wrows = kTiles * p.n_out;

  // First position at or after segment s; (seg, base) with base >= hi: the end.
  auto enter = [&](MfIter& it, int s) {
    it.seg = s;
    it.base = max(lo, s * nb);
    it.end = min(hi, (s + 1) * nb);
    it.c = c0;
  };
  // Next item.  A warp without a block in a round has one empty item there.
  auto step = [&](MfIter& it) -> bool {   // true: the round ended
    if (it.base + my_block < it.end && ++it.c < c1) return false;
    it.base += per_round;
    it.c = c0;
    if (it.base >= it.end && it.end < hi) enter(it, it.seg + 1);
    return true;
  };

  MfIter ld;
  const uint8_t* wptr = nullptr;   // this lane's first byte of row g of the loader's tile
  bool ok_lo = false, ok_hi = false;
  auto set_tile = [&]() {
    const int b = ld.base + my_block;
    ok_lo = ok_hi = false;
    if (ld.base < hi && b < ld.end) {
      const int n0 = (b - ld.seg * nb) * 16 + g;   // this lane's output rows n0 and n0 + 8
      ok_lo = n0 < p.n_out;
      ok_hi = n0 + 8 < p.n_out;
      wptr = p.w + (static_cast<int64_t>(mf_seg_expert(segs[ld.seg])) * wrows + sub * p.n_out + n0) * p.K + 16 * t4;
    }
  };
  const uint32_t ring_lane = smem_u32(ring) + lane * 16;
  auto issue = [&](int slot) {
    if (ld.base < hi) {
      const uint32_t dst = ring_lane + slot * kMfPieceBytes;
      const int k = ld.c * kMfChunk + 16 * t4;
      const bool k0 = k < p.K, k1 = k + 64 < p.K;
      const uint8_t* src = wptr + ld.c * kMfChunk;
      const uint8_t* src8 = src + static_cast<int64_t>(8) * p.K;
      if (ok_lo) {   // (outputs past the end are neither loaded nor stored)
        cp_async_16_zfill(dst, k0 ? src : p.w, k0 ? 16u : 0u);
        cp_async_16_zfill(dst + 1024, k1 ? src + 64 : p.w, k1 ? 16u : 0u);
      }
      if (ok_hi) {
        cp_async_16_zfill(dst + 512, k0 ? src8 : p.w, k0 ? 16u : 0u);
        cp_async_16_zfill(dst + 1536, k1 ? src8 + 64 : p.w, k1 ? 16u : 0u);
      }
      if (step(ld)) set_tile();
    }
    cp_async_commit();
  };
  int slot_ld = 0, slot = 0;
  if (lo < hi) {
    enter(ld, lo / nb);
    set_tile();
  } else {
    ld.base = hi;
  }
#pragma unroll
  for (int i = 0; i < kDepth - 1; ++i) issue(slot_ld++);
  slot_ld = kDepth - 1;

  if (!kUp) {
    pdl_wait_prior_grid();
    pdl_launch_dependents();
  }

  MfIter it;
  if (lo < hi) enter(it, lo / nb);
  int buf = 0;
  for (int s = lo < hi ? lo / nb : nseg; s * nb < hi; ++s) {
    const int seg = segs[s];
    const int cnt = mf_seg_count(seg);
    const int nt = (cnt + 7) >> 3;
    const int units = mf_part_units(NT);
    const bool two = 2 * nt <= units;   // two partial buffers fit: one barrier a round
    __syncthreads();                    // the codes and partials of the segment before are done with
    mf_build_rows<kUp>(p, seg, rows, codes, L.pitch, scales, warp, lane);
    __syncthreads();
    const uint8_t* brow = codes + g * L.pitch + 16 * t4;
    const int base0 = it.base, end = it.end;
    for (int base = base0; base < end; base += per_round) {
      const bool mine = base + my_block < end;
      float acc[NT][4];
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.0f;
      for (int c = c0; c < (mine ? c1 : c0 + 1); ++c) {
        cp_async_wait_group<kDepth - 2>();
        if (mine) {
          const uint32_t src = ring_lane + slot * kMfPieceBytes;
          const uint4 l0 = ld_shared_v4(src), h0 = ld_shared_v4(src + 512);
          const uint4 l1 = ld_shared_v4(src + 1024), h1 = ld_shared_v4(src + 1536);
          const uint32_t b0 = smem_u32(brow + c * kMfChunk);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            if (j < nt) {
              const uint4 v0 = ld_shared_v4(b0 + j * 8 * L.pitch);
              mma_e4m3_m16n8k32(acc[j], l0.x, h0.x, l0.y, h0.y, v0.x, v0.y);
              mma_e4m3_m16n8k32(acc[j], l0.z, h0.z, l0.w, h0.w, v0.z, v0.w);
              const uint4 v1 = ld_shared_v4(b0 + j * 8 * L.pitch + 64);
              mma_e4m3_m16n8k32(acc[j], l1.x, h1.x, l1.y, h1.y, v1.x, v1.y);
              mma_e4m3_m16n8k32(acc[j], l1.z, h1.z, l1.w, h1.w, v1.z, v1.w);
            }
          }
        }
        issue(slot_ld);
        if (++slot == kDepth) slot = 0;
        if (++slot_ld == kDepth) slot_ld = 0;
      }
      // partial sums of the round, then the outputs
      float* pb = part + (two ? buf : 0) * nt * kMfWarps * 128;
      if (!two && base != base0) __syncthreads();   // the round before has been read
      if (mine) {
        float* dst = pb + warp * nt * 128 + g * 8 + 2 * t4;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          if (j < nt) {
            *reinterpret_cast<float2*>(dst + j * 128) = make_float2(acc[j][0], acc[j][1]);
            *reinterpret_cast<float2*>(dst + j * 128 + 64) = make_float2(acc[j][2], acc[j][3]);
          }
        }
      }
      __syncthreads();
      const int e = mf_seg_expert(seg), row0 = mf_seg_row0(seg);
      const int blocks = min(per_round, end - base);
      for (int i = threadIdx.x; i < blocks * cnt * 16; i += kMfThreads) {
        const int u = i & 15, br = i >> 4;
        const int r = br % cnt, b = br / cnt;
        const int n = (base + b - s * nb) * 16 + u;
        if (n >= p.n_out) continue;
        float z[kTiles];
#pragma unroll
        for (int q = 0; q < kTiles; ++q) {
          const float* src = pb + (b * kTiles + q) * S * nt * 128 + (r >> 3) * 128 + u * 8 + (r & 7);
          float v = 0.0f;
          for (int k = 0; k < S; ++k) v = __fadd_rn(v, src[k * nt * 128]);
          z[q] = __fmul_rn(__fmul_rn(v, scales[r]),
                           __ldg(p.s_w + static_cast<int64_t>(e) * wrows + q * p.n_out + n));
        }
        const int64_t at = static_cast<int64_t>(rows[row0 + r]) * p.n_out + n;
        if (kUp) {
          float h = activate(z[0], p.act);
          if (kGated) h = __fmul_rn(h, z[kTiles - 1]);
          p.hidden[at] = __float2half_rn(h);
        } else {
          p.y[at] = z[0];
        }
      }
      buf ^= 1;
    }
    if (end < hi) enter(it, s + 1);
  }
  cp_async_wait_group<0>();
}

// out[t] = fp16(sum over the token's experts of weight * y + residual).
__global__ void __launch_bounds__(256) moe_few_combine_kernel(const float* y, const int32_t* experts,
                                                              const float* weights, const __half* residual, int T,
                                                              int topk, int E, int N, __half* out) {
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  const int n4 = N >> 2;
  for (int i = blockIdx.x * 256 + threadIdx.x; i < T * n4; i += gridDim.x * 256) {
    const int t = i / n4, c = (i - t * n4) * 4;
    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int j = 0; j < topk; ++j) {
      const int e = __ldg(experts + t * topk + j);
      if (e < 0 || e >= E) continue;
      const float w = __ldg(weights + t * topk + j);
      const float4 v = *reinterpret_cast<const float4*>(y + static_cast<int64_t>(t * topk + j) * N + c);
      a.x = fmaf(w, v.x, a.x);
      a.y = fmaf(w, v.y, a.y);
      a.z = fmaf(w, v.z, a.z);
      a.w = fmaf(w, v.w, a.w);
    }
    const int64_t at = static_cast<int64_t>(t) * N + c;
    if (residual != nullptr) {
      const __half2* r = reinterpret_cast<const __half2*>(residual + at);
      const float2 r0 = __half22float2(r[0]), r1 = __half22float2(r[1]);
      a.x += r0.x;
      a.y += r0.y;
      a.z += r1.x;
      a.w += r1.y;
    }
    __half2 h[2] = {__floats2half2_rn(a.x, a.y), __floats2half2_rn(a.z, a.w)};
    *reinterpret_cast<uint2*>(out + at) = *reinterpret_cast<const uint2*>(h);
  }
}

}  // namespace fp8q
