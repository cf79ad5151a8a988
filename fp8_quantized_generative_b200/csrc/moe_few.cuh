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
// is a run of units of `outs` outputs (RU = 16, 32 or 64 weight rows; gated: half of
// them from each half of the up projection).  Every CTA takes an equal share of
// the units of all segments.  One warp streams the weights with TMA (boxes of 128
// bytes of K x the unit's rows, 128-byte swizzle) through a ring of 32 KB stages, as
// far ahead of eight consumer warps as the ring reaches, across unit and segment
// boundaries.  For a segment the consumers first quantize its rows into shared
// memory; then S = 128 / RU of them share a 16-row tile's K, 256 bytes each a stage.
// K may be permuted in a product as long as both operands agree: lane (g, t) holds
// bytes 16 t .. 16 t + 15 of a 64-byte group of row g, which is one 16-byte shared
// load per row for two MMAs, for both operands.  The S partial sums of a tile
// meet in shared memory and are added in fixed order.
#pragma once

#include <cuda.h>

#include "activation.cuh"
#include "quant_rows.cuh"

namespace fp8q {

constexpr int kMfWarps = 8;                          // consumer warps
constexpr int kMfConsumers = kMfWarps * 32;
constexpr int kMfThreads = kMfConsumers + 32;        // + the warp that streams the weights
constexpr int kMfMaxRows = 1024;       // T * topk
constexpr int kMfMaxTopk = 8;
constexpr int kMfMaxExperts = 1024;
constexpr int kMfWarpK = 256;          // K bytes a warp takes of a stage
constexpr int kMfStageBytes = 32768;   // RU weight rows x 256 S bytes, S = 128 / RU
constexpr int kMfMaxStages = 6;
constexpr int kMfMaxSmem = 232448;     // 227 KB

struct MoeFewParams {
  const __half* x;          // up: [T, K]; down: hidden [T * topk, K]
  const int32_t* experts;   // [T * topk], -1: none
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
  int ru;                   // weight rows of a unit: 16, 32 or 64 (gated: 32 or 64)
  int stages;               // of the ring
};

// Shared-memory layout, the same on host and device.
struct MoeFewLayout {
  int pitch;      // bytes of a row of codes
  int codes;      // offsets
  int part;
  int scales;
  int bars;
  int rows;
  int segs;
  int counts;
  int total;
};
__host__ __device__ constexpr int mf_part_units(int nt) { return nt >= 4 ? 8 : 2 * nt; }   // x 4 KB
__host__ __device__ inline MoeFewLayout mf_layout(int nt, int K, int rmax, int stages, int R, int E) {
  MoeFewLayout l;
  l.pitch = (K + 127) / 128 * 128 + 64;
  l.codes = stages * kMfStageBytes;                    // the ring comes first (swizzle atoms: 1 KB aligned)
  l.part = l.codes + rmax * l.pitch;
  l.scales = l.part + mf_part_units(nt) * kMfWarps * 512;
  l.bars = l.scales + (64 + kMfWarps) * 4;             // row scales, then the build's partial maxima
  l.rows = l.bars + (2 * kMfMaxStages + 1) * 8;        // full, empty; the last word: abort flag
  l.segs = l.rows + R * 4;
  l.counts = l.segs + R * 4;
  l.total = l.counts + (E + 4) * 4;
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

// Consumer warps: quantize the rows of a segment into shared memory (codes
// [cnt][pitch], zero behind K; scales).  With few rows several warps share one
// (their maxima meet in `maxima`), so that a row's loads are all in flight at once.
template <bool kUp>
__device__ __forceinline__ void mf_build_rows(const MoeFewParams& p, int seg, const int* rows, uint8_t* codes,
                                              int pitch, float* scales, float* maxima, int warp, int lane) {
  constexpr int kHeld = 8;   // 16-byte vectors a lane keeps between the maximum and the codes
  const int cnt = mf_seg_count(seg), row0 = mf_seg_row0(seg);
  const int share = cnt > 4 ? 1 : cnt > 2 ? 2 : cnt > 1 ? 4 : 8;   // warps of a row
  const int nvec = p.K >> 3;
  const int nvec_pad = (pitch - 64) >> 3;
  const int j0 = (warp % share) * 32 + lane, step = share * 32;
  for (int i0 = 0; i0 < cnt; i0 += kMfWarps / share) {
    const int i = i0 + warp / share;
    const bool live = i < cnt;
    const uint4* src = nullptr;
    uint4 v[kHeld];
    float m = 0.0f;
    if (live) {
      const int slot = rows[row0 + i];
      src = reinterpret_cast<const uint4*>(p.x + static_cast<int64_t>(kUp ? slot / p.topk : slot) * p.K);
#pragma unroll
      for (int u = 0; u < kHeld; ++u)
        v[u] = j0 + u * step < nvec ? ld_global_v4(src + j0 + u * step) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int u = 0; u < kHeld; ++u) m = absmax8(v[u], m);
      for (int j = j0 + kHeld * step; j < nvec; j += step) m = absmax8(ld_global_v4(src + j), m);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    if (share > 1) {   // uniform; one pass over the rows in this case
      if (lane == 0) maxima[warp] = m;
      named_barrier(1, kMfConsumers);
      for (int k = 0; k < share; ++k) m = fmaxf(m, maxima[warp / share * share + k]);
    }
    if (live) {
      const RowScale rs = row_scale_from_amax(m);
      uint2* dst = reinterpret_cast<uint2*>(codes + i * pitch);
#pragma unroll
      for (int u = 0; u < kHeld; ++u)   // (vectors behind K are zero: zero codes)
        if (j0 + u * step < nvec_pad) dst[j0 + u * step] = encode8(v[u], rs.r);
      for (int j = j0 + kHeld * step; j < nvec_pad; j += step)
        dst[j] = j < nvec ? encode8(ld_global_v4(src + j), rs.r) : make_uint2(0u, 0u);
      if (j0 == 0) scales[i] = rs.s;
    }
  }
}

// NT: n-tiles of 8 rows a segment may have.  tmW: the weights [E * wrows, K] in
// boxes of 128 bytes x RU rows (gated: RU / 2).
template <int NT, bool kUp, bool kGated>
__global__ void __launch_bounds__(kMfThreads) moe_few_kernel(const __grid_constant__ CUtensorMap tmW,
                                                             const MoeFewParams p) {
  extern __shared__ __align__(1024) uint8_t mf_smem[];
  constexpr int kHalves = kUp && kGated ? 2 : 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const MoeFewLayout L = mf_layout(NT, p.K, p.rmax, p.stages, p.rows, p.E);
  uint8_t* ring = mf_smem;
  uint8_t* codes = mf_smem + L.codes;
  float* part = reinterpret_cast<float*>(mf_smem + L.part);
  float* scales = reinterpret_cast<float*>(mf_smem + L.scales);
  uint64_t* full = reinterpret_cast<uint64_t*>(mf_smem + L.bars);
  uint64_t* empty = full + kMfMaxStages;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(empty + kMfMaxStages);
  int* rows = reinterpret_cast<int*>(mf_smem + L.rows);
  int* segs = reinterpret_cast<int*>(mf_smem + L.segs);
  int* counts = reinterpret_cast<int*>(mf_smem + L.counts);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kMfMaxStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kMfWarps);
    }
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tmap(&tmW);
  }
  // The experts may come from the kernel just before the up projection.  The
  // down projection starts once every CTA of the up projection has passed this
  // wait, so the experts are there and only the hidden rows are waited for.
  if (kUp) {
    pdl_wait_prior_grid();
    pdl_launch_dependents();
  }
  const int nseg = mf_schedule(p, rows, segs, counts, reinterpret_cast<int*>(part), kUp && blockIdx.x == 0);
  const int outs = p.ru / kHalves;                  // outputs of a unit
  const int nu = (p.n_out + outs - 1) / outs;       // units of a segment
  const int total = nseg * nu;
  const int lo = static_cast<int>(static_cast<int64_t>(total) * blockIdx.x / gridDim.x);
  const int hi = static_cast<int>(static_cast<int64_t>(total) * (blockIdx.x + 1) / gridDim.x);
  const int S = 128 / p.ru;                         // warps that share a tile's K
  const int boxes = (p.K + 127) / 128;              // 128-byte boxes of K
  const int stage_boxes = 2 * S;
  const int wrows = kHalves * p.n_out;

  if (warp == kMfWarps) {
    // ------------------------------------------------------------ weights
    if (lane == 0) {
      int slot = 0;
      uint32_t ph = 0, armed = 0, armed_ph = 0;
      bool ok = true;
      int s = lo < hi ? lo / nu : 0;
      int n0 = (lo - s * nu) * outs;
      for (int i = lo; i < hi && ok; ++i) {
        const int row = mf_seg_expert(segs[s]) * wrows + n0;
        for (int b0 = 0; b0 < boxes; b0 += stage_boxes) {
          const int nbox = min(stage_boxes, boxes - b0);
          if (!mbar_wait(&empty[slot], ph ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[slot], static_cast<uint32_t>(nbox * p.ru * 128));
          uint8_t* dst = ring + slot * kMfStageBytes;
          for (int b = 0; b < nbox; ++b) {
#pragma unroll
            for (int q = 0; q < kHalves; ++q) {
              tma_load_2d(dst, &tmW, &full[slot], (b0 + b) * 128, row + q * p.n_out);
              dst += outs * 128;
            }
          }
          armed |= 1u << slot;
          armed_ph = (armed_ph & ~(1u << slot)) | (ph << slot);
          if (++slot == p.stages) {
            slot = 0;
            ph ^= 1u;
          }
        }
        n0 += outs;
        if (n0 >= p.n_out) {
          n0 = 0;
          ++s;
        }
      }
      if (!ok) {
        raise_error(0x1u);
        *abort_flag = 1;
      }
      // No copy may still be in flight when the CTA exits.
      for (int i = 0; i < p.stages; ++i)
        if (armed & (1u << i)) mbar_wait(&full[i], (armed_ph >> i) & 1u, nullptr);
    }
    return;
  }

  // -------------------------------------------------------------- consumers
  const int g = lane >> 2, t4 = lane & 3;
  const int ks = warp % S, tl = warp / S;           // share of K, 16-row tile of the unit
  if (!kUp) {
    pdl_wait_prior_grid();
    pdl_launch_dependents();
  }
  int slot = 0, buf = 0;
  uint32_t ph = 0;
  for (int s = lo < hi ? lo / nu : nseg; s * nu < hi; ++s) {
    const int seg = segs[s];
    const int e = mf_seg_expert(seg), cnt = mf_seg_count(seg), row0 = mf_seg_row0(seg);
    const int nt = (cnt + 7) >> 3;
    const bool two = 2 * nt <= mf_part_units(NT);   // two partial buffers fit: one barrier a unit
    named_barrier(1, kMfConsumers);                 // the codes and partials of the segment before are done with
    mf_build_rows<kUp>(p, seg, rows, codes, L.pitch, scales, scales + 64, warp, lane);
    named_barrier(1, kMfConsumers);
    const uint32_t brow = smem_u32(codes + g * L.pitch + 16 * t4);
    const int first = max(lo, s * nu), end = min(hi, (s + 1) * nu);
    for (int unit = first; unit < end; ++unit) {
      const int n0 = (unit - s * nu) * outs;
      // the weight scales of this thread's first output, in flight during the mainloop
      const int u = threadIdx.x & (outs - 1), r1 = threadIdx.x / outs;
      const float* sw = p.s_w + static_cast<int64_t>(e) * wrows + n0 + u;
      const bool live = n0 + u < p.n_out;
      float w[kHalves];
#pragma unroll
      for (int q = 0; q < kHalves; ++q) w[q] = live ? __ldg(sw + q * p.n_out) : 0.0f;
      float acc[NT][4];
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.0f;
      for (int b0 = 0; b0 < boxes; b0 += stage_boxes) {
        if (!mbar_wait(&full[slot], ph, abort_flag)) {
          // give up, but walk on: every warp meets the same barriers
          if (lane == 0) raise_error(0x4u);
          *abort_flag = 1;
        }
        const uint32_t arow = smem_u32(ring + slot * kMfStageBytes) + (tl * 16 + g) * 128;
#pragma unroll
        for (int h = 0; h < 4; ++h) {   // 64-byte groups of this warp's two boxes
          const int box = 2 * ks + (h >> 1);
          if (b0 + box < boxes) {
            // 16-byte chunk c of a row lies at chunk c ^ (row & 7)
            const uint32_t at = arow + box * p.ru * 128 + ((((h & 1) * 4 + t4) ^ g) << 4);
            const uint4 a = ld_shared_v4(at), b = ld_shared_v4(at + 8 * 128);
            const uint32_t xrow = brow + (b0 + box) * 128 + (h & 1) * 64;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              if (j < nt) {
                const uint4 x = ld_shared_v4(xrow + j * 8 * L.pitch);
                mma_e4m3_m16n8k32(acc[j], a.x, b.x, a.y, b.y, x.x, x.y);
                mma_e4m3_m16n8k32(acc[j], a.z, b.z, a.w, b.w, x.z, x.w);
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[slot]);
        if (++slot == p.stages) {
          slot = 0;
          ph ^= 1u;
        }
      }
      // partial sums of the unit, then its outputs
      float* pb = part + (two ? buf : 0) * nt * kMfWarps * 128;
      if (!two && unit != first) named_barrier(1, kMfConsumers);   // the unit before has been read
      float* dst = pb + warp * nt * 128 + g * 8 + 2 * t4;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if (j < nt) {
          *reinterpret_cast<float2*>(dst + j * 128) = make_float2(acc[j][0], acc[j][1]);
          *reinterpret_cast<float2*>(dst + j * 128 + 64) = make_float2(acc[j][2], acc[j][3]);
        }
      }
      named_barrier(1, kMfConsumers);
      for (int r = r1; r < cnt && live; r += kMfConsumers / outs) {
        float z[kHalves];
#pragma unroll
        for (int q = 0; q < kHalves; ++q) {
          const int tile = q * (outs / 16) + (u >> 4);
          const float* src = pb + tile * S * nt * 128 + (r >> 3) * 128 + (u & 15) * 8 + (r & 7);
          float v = 0.0f;
          for (int k = 0; k < S; ++k) v = __fadd_rn(v, src[k * nt * 128]);
          z[q] = __fmul_rn(__fmul_rn(v, scales[r]), w[q]);
        }
        const int64_t at = static_cast<int64_t>(rows[row0 + r]) * p.n_out + n0 + u;
        if (kUp) {
          float h = activate(z[0], p.act);
          if (kGated) h = __fmul_rn(h, z[kHalves - 1]);
          p.hidden[at] = __float2half_rn(h);
        } else {
          p.y[at] = z[0];
        }
      }
      buf ^= 1;
    }
  }
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
