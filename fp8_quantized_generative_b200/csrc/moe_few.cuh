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
// streaming the chosen experts' weights once from HBM: 23 bytes a cycle and SM, a 32 KB
// stage in 1400 cycles.  16 weight rows are the M operand of an MMA and up to 8
// rows an n-tile.  The codes of both operands become fp16 (exact) and go through
// mma.sync m16n8k16 with fp32 accumulators: its E4M3 form, without the conversions, was
// measured at 1110 cycles for the products of a stage where this form takes 650 to 740,
// so that the stage's HBM time hides it.  A tcgen05 tile
// would read FP8 itself, but wants 64 or 128 weight rows to a tile, too coarse to
// spread one token's experts over 148 SMs, and its issue takes 26-42 ns per 32 bytes
// of K whatever the row count: 1.7 us and more on the one chain of K = 2048 that
// eight warps share here.
//
// Work: the chosen experts, each cut into segments of at most rmax rows; a segment
// is a run of units of `outs` outputs (RU = 16, 32 or 64 weight rows; gated: half of
// them from each half of the up projection).  Every CTA takes an equal share of
// the units of all segments, where a segment's start counts as so many units more as
// its quantization costs.  Its warps:
//   0..7    quantize a segment's rows into shared memory, then multiply: each takes
//           an eighth of a stage's K for all rows of the unit and leaves its partial
//           sums of the unit in shared memory;
//   8..11   add the eight partial sums in fixed order, scale, activate, store, while
//           the multiplying warps are at the next unit;
//   12      streams the weights with TMA (boxes of 128 bytes of K x the unit's rows,
//           128-byte swizzle) through a ring of 32 KB stages, as far ahead as the
//           ring reaches, across unit and segment boundaries.
// Both operands reach the MMA through ldmatrix (16-byte row pieces; the weights'
// swizzle and a pitch of 16 bytes off a multiple of 128 for the rows keep the eight
// rows of a matrix on different banks).  K may be permuted in a product as long as both
// operands agree: of a 16-byte piece of weights, lane (g, t) holds bytes 4 t .. 4 t + 3
// of row g, which converted are the two K pairs of one MMA, so the fp16 rows are
// stored with the pairs of every 16 values in the order 0 2 4 6 1 3 5 7.
#pragma once

#include <cuda.h>

#include "activation.cuh"
#include "quant_rows.cuh"

namespace fp8q {

constexpr int kMfWarps = 8;                          // quantize and multiply
constexpr int kMfConsumers = kMfWarps * 32;
constexpr int kMfEpiWarps = 4;                       // partial sums to outputs
constexpr int kMfEpiThreads = kMfEpiWarps * 32;
constexpr int kMfThreads = kMfConsumers + kMfEpiThreads + 32;   // + the warp that streams the weights
constexpr int kMfMaxRows = 1024;       // T * topk
constexpr int kMfMaxTopk = 8;
constexpr int kMfMaxExperts = 1024;
static_assert(kMfMaxRows <= 1024 && kMfMaxExperts <= 1024, "rows and experts are packed in 10 bits each (mf_seg, mf_schedule)");
constexpr int kMfFuseTokens = 16;      // and units a CTA of the down projection, at most,
constexpr int kMfFuseUnits = 3;        // for it to add the rows up
constexpr int kMfStageBytes = 32768;   // RU weight rows x 32 KB / RU of K
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
  // With few tokens and few units a CTA the down projection also adds the tokens'
  // rows up (done != nullptr); else moe_few_combine_kernel does.
  uint32_t* done;           // a counter a unit of the down projection, zeroed by the up projection
  int done_units;
  const float* weights;     // [T * topk]
  const __half* residual;   // [T, N] or nullptr
  __half* out;              // [T, N]
  int rmax;                 // rows of a segment, a multiple of 8
  int units;                // of a segment
  int lead;                 // places before a segment's units that stand for its quantization in the equal shares
  int stages;               // of the ring
};

// Shared-memory layout, the same on host and device.
struct MoeFewLayout {
  int pitch;      // bytes of a quantized row (fp16 values of its codes)
  int codes;      // offsets
  int part;
  int scales;
  int bars;
  int rows;
  int segs;
  int counts;
  int total;
};
// Partial sums of a unit: mt weight tiles x nt n-tiles x 8 warps, 512 bytes each.
__host__ __device__ constexpr int mf_part_bufs(int nt, int mt) { return nt * mt > 4 ? 1 : 2; }
__host__ __device__ inline MoeFewLayout mf_layout(int nt, int mt, int K, int rmax, int stages, int R, int E) {
  MoeFewLayout l;
  l.pitch = (K + 127) / 128 * 256 + 16;
  l.codes = stages * kMfStageBytes;                    // the ring comes first (swizzle atoms: 1 KB aligned)
  l.part = l.codes + rmax * l.pitch;
  l.scales = l.part + mf_part_bufs(nt, mt) * nt * mt * kMfWarps * 512;
  l.bars = l.scales + (3 * 64 + kMfWarps) * 4;         // row scales of three segments, the build's partial maxima
  l.rows = l.bars + (2 * kMfMaxStages + 5) * 8;        // full, empty, partials full [2] / empty [2], abort flag
  l.segs = l.rows + R * 4;
  l.counts = l.segs + R * 4;
  l.total = l.counts + (E + 4) * 4;
  return l;
}

__device__ __forceinline__ void mma_f16_m16n8k16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four E4M3 codes -> fp16 pairs (exact): codes 0, 1 and codes 2, 3.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t v, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(v));
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// One segment: expert (10 bits) | rows - 1 (6) | first entry in the row list (10).
__device__ __forceinline__ int mf_seg(int e, int cnt, int row0) { return e | (cnt - 1) << 10 | row0 << 16; }
__device__ __forceinline__ int mf_seg_expert(int s) { return s & 1023; }
__device__ __forceinline__ int mf_seg_count(int s) { return ((s >> 10) & 63) + 1; }
__device__ __forceinline__ int mf_seg_row0(int s) { return s >> 16; }

// Group the rows by expert: segs[] and the row list (slots by expert).  Within an
// expert that fits one segment the rows lie in the order of the atomics, which only
// decides the column of an MMA that a row takes; where an expert is cut, they
// are put in ascending order, so that all CTAs that share it cut it alike.
// Up to 32 rows, where the start is most of the time, one warp does it all without
// the counters (one token 12.2 -> 11.1 us, 8 tokens with 4 choices 34.0 -> 33.2).
// ex: [rows] ints of scratch.  Returns the number of segments.
__device__ __forceinline__ int mf_schedule(const MoeFewParams& p, int* rows, int* segs, int* counts, int* ex,
                                           bool report) {
  const int tid = threadIdx.x;
  if (p.rows <= 32) {   // one warp, a lane a row; segments in the order of their first rows
    if (tid < 32) {
      int e = tid < p.rows ? __ldg(p.experts + tid) : -1;
      if (e < -1 || e >= p.E) {
        if (report) raise_error(0x8u);
        e = -1;
      }
      const uint32_t same = __match_any_sync(0xffffffffu, e);   // rows of the same expert
      const int rank = __popc(same & ((1u << tid) - 1u));
      const int c = e >= 0 && rank == 0 ? __popc(same) : 0;
      const int mine = c | ((c + p.rmax - 1) / p.rmax) << 16;
      int at = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, at, o);
        if (tid >= o) at += v;
      }
      if (tid == 31) counts[p.E] = at >> 16;
      at -= mine;
      const int r0 = __shfl_sync(0xffffffffu, at & 0xffff, __ffs(same) - 1);
      if (e >= 0) rows[r0 + rank] = tid;
      int s0 = at >> 16;
      for (int k = 0; k < c; k += p.rmax) segs[s0++] = mf_seg(e, min(p.rmax, c - k), r0 + k);
    }
    __syncthreads();
    return counts[p.E];
  }
  for (int e = tid; e <= p.E; e += kMfThreads) counts[e] = 0;
  __syncthreads();
  for (int r = tid; r < p.rows; r += kMfThreads) {
    const int e = __ldg(p.experts + r);
    int v = -1;
    if (e >= 0 && e < p.E) v = e | atomicAdd(&counts[e], 1) << 10;
    else if (e != -1 && report) raise_error(0x8u);
    ex[r] = v;   // expert and place within it
  }
  __syncthreads();
  if (tid < 32) {
    const int per = (p.E + 31) >> 5;
    const int e0 = min(p.E, tid * per), e1 = min(p.E, e0 + per);
    int nr = 0, ns = 0, cut = 0;
    for (int e = e0; e < e1; ++e) {
      const int c = counts[e];
      nr += c;
      ns += c <= p.rmax ? (c > 0) : (c + p.rmax - 1) / p.rmax;
      cut |= c > p.rmax;
    }
    int at = nr | ns << 16;   // both at most 1024: one scan
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, at, o);
      if (tid >= o) at += v;
    }
    int r0 = (at & 0xffff) - nr, s0 = (at >> 16) - ns;
    for (int e = e0; e < e1; ++e) {
      const int c = counts[e];
      counts[e] = r0;   // from here on: the expert's first entry in the row list
      for (int k = 0; k < c; k += p.rmax) segs[s0++] = mf_seg(e, min(p.rmax, c - k), r0 + k);
      r0 += c;
    }
    if (tid == 31) counts[p.E] = at >> 16;
    cut = __any_sync(0xffffffffu, cut);
    if (cut) {   // ascending places, 32 rows at a time
      for (int r = tid; r - tid < p.rows; r += 32) {
        const int e = r < p.rows ? (ex[r] < 0 ? -1 : ex[r] & 1023) : -1;
        const uint32_t same = __match_any_sync(0xffffffffu, e);
        const int first = e >= 0 ? counts[e] : 0;
        __syncwarp();
        if (e >= 0) {
          const int rank = __popc(same & ((1u << tid) - 1u));
          rows[first + rank] = r;
          ex[r] = -1;
          if (rank == 0) counts[e] = first + __popc(same);
        }
        __syncwarp();
      }
    }
  }
  __syncthreads();
  for (int r = tid; r < p.rows; r += kMfThreads) {
    const int v = ex[r];
    if (v >= 0) rows[counts[v & 1023] + (v >> 10)] = r;
  }
  __syncthreads();
  return counts[p.E];
}

// max(m, |x|) of eight fp16 values, two maxima side by side (exact: no rounding).
__device__ __forceinline__ __half2 absmax8_f16(const uint4& v, __half2 m) {
  const __half2* h = reinterpret_cast<const __half2*>(&v);
  return __hmax2(__hmax2(m, __hmax2(__habs2(h[0]), __habs2(h[1]))), __hmax2(__habs2(h[2]), __habs2(h[3])));
}

// Four fp16 values -> the fp16 values of their codes.
__device__ __forceinline__ uint2 quantize4_f16(const uint2& v, float r) {
  const __half2* h = reinterpret_cast<const __half2*>(&v);
  const float2 f0 = __half22float2(h[0]), f1 = __half22float2(h[1]);
  const uint32_t c = static_cast<uint32_t>(cvt_e4m3x2(__fmul_rn(f0.x, r), __fmul_rn(f0.y, r))) |
                     static_cast<uint32_t>(cvt_e4m3x2(__fmul_rn(f1.x, r), __fmul_rn(f1.y, r))) << 16;
  uint2 o;
  e4m3x4_to_f16(c, o.x, o.y);
  return o;
}

// Quantize the rows of a segment into shared memory (the fp16 values of the codes
// [cnt][pitch], zero behind K, pairs permuted as above; scales).  A lane first
// copies its 16-byte pieces of the row to where their codes will lie, kLoads loads in
// flight, with the maximum on the way, and then converts them in place: one read
// from global for any K, in little code (the kernel starts cold).  With few rows
// several warps share one; their maxima meet in `maxima`.  kLoads: eight where a CTA
// has many units and starts segments while its weights stream, four where the start is
// most of the time (one token of 64 experts, 2048-1024-2048, 12.8 -> 12.2 us for the
// layer; 64 tokens with four 49.3 -> 53.0).
template <bool kUp, int kLoads>
__device__ __forceinline__ void mf_build_rows(const MoeFewParams& p, int seg, const int* rows, uint8_t* codes,
                                              int pitch, float* scales, float* maxima, int warp, int lane) {
  const int cnt = mf_seg_count(seg), row0 = mf_seg_row0(seg);
  const int share_log = cnt > 4 ? 0 : cnt > 2 ? 1 : cnt > 1 ? 2 : 3;   // 2^share_log warps of a row
  const int nvec = p.K >> 3;
  const int nvec_pad = (pitch - 16) >> 4;
  const int j0 = (warp & ((1 << share_log) - 1)) * 32 + lane, step = 32 << share_log;
  for (int i0 = 0; i0 < cnt; i0 += kMfWarps >> share_log) {
    const int i = i0 + (warp >> share_log);
    const bool live = i < cnt;
    // piece j of the row: values 8 j .. 8 j + 7, at its 32-byte group's halves
    uint8_t* dst = codes + i * pitch + (j0 >> 1) * 32 + (j0 & 1) * 8;
    float m = 0.0f;
    if (live) {
      const int slot = rows[row0 + i];
      const uint4* src = reinterpret_cast<const uint4*>(p.x + static_cast<int64_t>(kUp ? slot / p.topk : slot) * p.K);
      __half2 m2 = __float2half2_rn(0.0f);
#pragma unroll 1
      for (int j = j0; j < nvec_pad; j += kLoads * step) {
        uint4 v[kLoads];
#pragma unroll
        for (int u = 0; u < kLoads; ++u)
          v[u] = j + u * step < nvec ? ld_global_v4(src + j + u * step) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
          m2 = absmax8_f16(v[u], m2);
          if (j + u * step < nvec_pad) {
            uint8_t* at = dst + (j - j0 + u * step) * 16;
            *reinterpret_cast<uint2*>(at) = make_uint2(v[u].x, v[u].z);
            *reinterpret_cast<uint2*>(at + 16) = make_uint2(v[u].y, v[u].w);
          }
        }
      }
      m = fmaxf(__low2float(m2), __high2float(m2));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    if (share_log > 0) {   // uniform; one pass over the rows in this case
      if (lane == 0) maxima[warp] = m;
      named_barrier(1, kMfConsumers);
      const int w0 = warp >> share_log << share_log;
      for (int k = 0; k < 1 << share_log; ++k) m = fmaxf(m, maxima[w0 + k]);
    }
    if (live) {
      const RowScale rs = row_scale_from_amax(m);
#pragma unroll 2
      for (int j = j0; j < nvec_pad; j += step) {
        uint2* at = reinterpret_cast<uint2*>(dst + (j - j0) * 16);
        const uint2 a = at[0], b = at[2];
        at[0] = quantize4_f16(a, rs.r);
        at[2] = quantize4_f16(b, rs.r);
      }
      if (j0 == 0) scales[i] = rs.s;
    }
  }
}

// The weighted sum of a token's rows, in the order of its choices, + residual, rounded once.
__device__ __forceinline__ void mf_add_weighted(float4& a, float w, const float4& v) {
  a.x = fmaf(w, v.x, a.x);
  a.y = fmaf(w, v.y, a.y);
  a.z = fmaf(w, v.z, a.z);
  a.w = fmaf(w, v.w, a.w);
}
__device__ __forceinline__ void mf_store_out(const __half* residual, __half* out, int64_t at, float4 a) {
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

// NT: n-tiles of 8 rows a segment may have; MT: 16-row weight tiles of a unit (RU =
// 16 MT).  tmW: the weights [E * wrows, K] in boxes of 128 bytes x RU rows (gated:
// RU / 2).
template <int NT, int MT, bool kUp, bool kGated>
__global__ void __launch_bounds__(kMfThreads) moe_few_kernel(const __grid_constant__ CUtensorMap tmW,
                                                             const MoeFewParams p) {
  extern __shared__ __align__(1024) uint8_t mf_smem[];
  constexpr int kHalves = kUp && kGated ? 2 : 1;
  constexpr int RU = 16 * MT;
  constexpr int outs = RU / kHalves;                // outputs of a unit
  static_assert(MT % kHalves == 0, "a gated unit has tiles of both halves");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const MoeFewLayout L = mf_layout(NT, MT, p.K, p.rmax, p.stages, p.rows, p.E);
  uint8_t* ring = mf_smem;
  uint8_t* codes = mf_smem + L.codes;
  float* part = reinterpret_cast<float*>(mf_smem + L.part);
  float* scales = reinterpret_cast<float*>(mf_smem + L.scales);
  uint64_t* full = reinterpret_cast<uint64_t*>(mf_smem + L.bars);
  uint64_t* empty = full + kMfMaxStages;
  uint64_t* pfull = empty + kMfMaxStages;
  uint64_t* pempty = pfull + 2;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(pempty + 2);
  volatile int* last_flag = abort_flag + 1;
  int* rows = reinterpret_cast<int*>(mf_smem + L.rows);
  int* segs = reinterpret_cast<int*>(mf_smem + L.segs);
  int* counts = reinterpret_cast<int*>(mf_smem + L.counts);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kMfMaxStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kMfWarps);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&pfull[b], kMfWarps);
      mbar_init(&pempty[b], kMfEpiWarps);
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
    if (p.done != nullptr && blockIdx.x == gridDim.x - 1)
      for (int i = threadIdx.x; i < p.done_units; i += kMfThreads) p.done[i] = 0;
  }
  const int nseg = mf_schedule(p, rows, segs, counts, reinterpret_cast<int*>(part), kUp && blockIdx.x == 0);
  const int nu = p.units;                           // units of a segment
  const int width = nu + p.lead;                    // places of a segment: its lead (no work), then its units
  const int total = nseg * width;
  const int share = total / static_cast<int>(gridDim.x), more = total - share * static_cast<int>(gridDim.x);
  const int lo = share * static_cast<int>(blockIdx.x) + min(static_cast<int>(blockIdx.x), more);
  const int hi = lo + share + (static_cast<int>(blockIdx.x) < more ? 1 : 0);
  const int s_first = lo < hi ? lo / width : nseg;  // first segment
  // units [first, end) of segment s in this share
  auto seg_first = [&](int s) { return max(lo - s * width - p.lead, 0); };
  auto seg_end = [&](int s) { return min(hi - s * width - p.lead, nu); };
  const int boxes = (p.K + 127) / 128;              // 128-byte boxes of K
  constexpr int stage_boxes = 16 / MT;
  const int wrows = kHalves * p.n_out;

  if (warp == kMfWarps + kMfEpiWarps) {
    // ------------------------------------------------------------ weights
    if (lane == 0) {
      int slot = 0;
      uint32_t ph = 0, armed = 0, armed_ph = 0;
      bool ok = true;
      for (int s = s_first; s * width < hi && ok; ++s) {
        const int end = seg_end(s);
        for (int unit = seg_first(s); unit < end && ok; ++unit) {
          const int row = mf_seg_expert(segs[s]) * wrows + unit * outs;
          for (int b0 = 0; b0 < boxes; b0 += stage_boxes) {
            const int nbox = min(stage_boxes, boxes - b0);
            if (!mbar_wait(&empty[slot], ph ^ 1u, abort_flag)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(&full[slot], static_cast<uint32_t>(nbox * RU * 128));
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

  constexpr int kBufs = mf_part_bufs(NT, MT);
  constexpr int kPartFloats = NT * MT * kMfWarps * 128;
  int buf = 0;
  uint32_t bph = 0;

  if (warp >= kMfWarps) {
    // ------------------------------------------------------------ partial sums to outputs
    // (the stores come after the wait below and the partials' first barrier: behind
    // the kernel before this one, as the multiplying warps wait for it)
    const int tid = threadIdx.x - kMfConsumers;
    // Adding up: this thread's first token and four columns of the unit, and what it
    // needs of the router, loaded ahead.
    constexpr bool kFuse = !kUp && NT <= 2;   // (more rows than that an expert: never fused)
    constexpr int kVec = outs / 4;
    const int tokens = p.rows / p.topk;
    float cw[kMfMaxTopk];
    uint32_t has = 0;   // choices with an expert
    auto load_choices = [&](int t) {
      has = 0;
#pragma unroll
      for (int j = 0; j < kMfMaxTopk; ++j) {
        if (j < p.topk) {
          const int e = __ldg(p.experts + t * p.topk + j);
          cw[j] = __ldg(p.weights + t * p.topk + j);
          has |= static_cast<uint32_t>(e >= 0 && e < p.E) << j;
        }
      }
    };
    if (kFuse && p.done != nullptr && tid < tokens * kVec) load_choices(tid / kVec);
    auto add_up = [&](int n0) {   // columns n0 .. n0 + outs - 1 of every token
#pragma unroll 1
      for (int i = tid; i < tokens * kVec; i += kMfEpiThreads) {
        const int t = i / kVec, n = n0 + (i % kVec) * 4;
        if (tokens * kVec > kMfEpiThreads) load_choices(t);   // (else every thread keeps its one token)
        if (n >= p.n_out) continue;
        const float* y = p.y + static_cast<int64_t>(t) * p.topk * p.n_out + n;
        float4 v[kMfMaxTopk];
#pragma unroll
        for (int j = 0; j < kMfMaxTopk; ++j)
          if (has >> j & 1u) v[j] = __ldcg(reinterpret_cast<const float4*>(y + static_cast<int64_t>(j) * p.n_out));
        float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int j = 0; j < kMfMaxTopk; ++j)
          if (has >> j & 1u) mf_add_weighted(a, cw[j], v[j]);
        mf_store_out(p.residual, p.out, static_cast<int64_t>(t) * p.n_out + n, a);
      }
    };
    constexpr int step = kMfEpiThreads / outs;
    const int u = tid & (outs - 1), r1 = tid / outs;
    for (int s = s_first, k3 = 0; s * width < hi; ++s) {
      const int first = seg_first(s), end = seg_end(s);
      if (first >= end) continue;
      const int seg = segs[s];
      const int e = mf_seg_expert(seg), cnt = mf_seg_count(seg), row0 = mf_seg_row0(seg);
      const int nt = (cnt + 7) >> 3;
      const float* sw = p.s_w + static_cast<int64_t>(e) * wrows + u;
      for (int unit = first; unit < end; ++unit) {
        const int n = unit * outs + u;
        const bool live = n < p.n_out;
        float w[kHalves];
#pragma unroll
        for (int q = 0; q < kHalves; ++q) w[q] = live ? __ldg(sw + q * p.n_out + n - u) : 0.0f;
        if (!mbar_wait(&pfull[buf], bph, abort_flag)) {
          if (lane == 0) raise_error(0x4u);
          *abort_flag = 1;
        }
        for (int r = r1; r < cnt && live; r += step) {
          float z[kHalves];
#pragma unroll
          for (int q = 0; q < kHalves; ++q) {
            const int tile = q * (outs >> 4) + (u >> 4);
            const float* src = part + buf * kPartFloats + (tile * nt + (r >> 3)) * 128 + (u & 15) * 8 + (r & 7);
            float v = src[0];   // in the order of K
#pragma unroll
            for (int k = 1; k < kMfWarps; ++k) v = __fadd_rn(v, src[k * MT * nt * 128]);
            z[q] = __fmul_rn(__fmul_rn(v, scales[k3 * 64 + r]), w[q]);
          }
          const int64_t at = static_cast<int64_t>(rows[row0 + r]) * p.n_out + n;
          if (kUp) {
            float h = activate(z[0], p.act);
            if (kGated) h = __fmul_rn(h, z[kHalves - 1]);
            p.hidden[at] = __float2half_rn(h);
          } else {
            p.y[at] = z[0];
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&pempty[buf]);
        if (++buf == kBufs) {
          buf = 0;
          bph ^= 1u;
        }
        if (kFuse && p.done != nullptr) {
          // the CTA that brings the last segment's rows of these columns adds them up
          named_barrier(3, kMfEpiThreads);
          if (tid == 0)
            *last_flag = atom_add_acq_rel_gpu(p.done + unit, 1u) == static_cast<uint32_t>(nseg - 1);
          named_barrier(3, kMfEpiThreads);
          if (*last_flag) add_up(n - u);
        }
      }
      k3 = k3 == 2 ? 0 : k3 + 1;
    }
    if (kFuse && p.done != nullptr && nseg == 0) {   // no token has an expert: residual or zero
      pdl_wait_prior_grid();
      for (int c = static_cast<int>(blockIdx.x) * outs; c < p.n_out; c += static_cast<int>(gridDim.x) * outs) add_up(c);
    }
    return;
  }

  // -------------------------------------------------------------- quantize and multiply
  if (!kUp) {
    pdl_wait_prior_grid();
    pdl_launch_dependents();
  }
  // ldmatrix rows of this lane: weights, row (lane & 15) and 16-byte piece lane >> 4
  // of a 32-byte group; fp16 rows, row lane & 7 and piece lane >> 3 of 64 bytes
  const uint32_t a_row = static_cast<uint32_t>((lane & 15) * 128);
  const uint32_t a_xor = static_cast<uint32_t>(lane & 7) << 4, a_piece = static_cast<uint32_t>(lane >> 4) << 4;
  const uint32_t b_row = smem_u32(codes) + (lane & 7) * L.pitch + ((lane >> 3) << 4);
  const int g = lane >> 2, t4 = lane & 3;
  int slot = 0;
  uint32_t ph = 0;
  bool codes_used = false;
  for (int s = s_first, k3 = 0; s * width < hi; ++s) {
    const int first = seg_first(s), end = seg_end(s);
    if (first >= end) continue;
    const int seg = segs[s];
    const int nt = (mf_seg_count(seg) + 7) >> 3;
    if (codes_used) named_barrier(1, kMfConsumers);   // the codes of the segment before are done with
    mf_build_rows<kUp, MT == 4 ? 8 : 4>(p, seg, rows, codes, L.pitch, scales + k3 * 64, scales + 3 * 64, warp, lane);
    named_barrier(1, kMfConsumers);
    codes_used = true;
    for (int unit = first; unit < end; ++unit) {
      // two accumulators a tile where few tiles keep the MMAs waiting for one another
      constexpr int kAcc = NT * MT <= 2 ? 2 : 1;
      float acc[MT][NT][kAcc][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int c = 0; c < kAcc; ++c) acc[m][j][c][0] = acc[m][j][c][1] = acc[m][j][c][2] = acc[m][j][c][3] = 0.0f;
      for (int b0 = 0; b0 < boxes; b0 += stage_boxes) {
        if (!mbar_wait(&full[slot], ph, abort_flag)) {
          // give up, but walk on: every warp meets the same barriers
          if (lane == 0) raise_error(0x4u);
          *abort_flag = 1;
        }
        const uint32_t stage = smem_u32(ring) + slot * kMfStageBytes + a_row;
        // This warp's 32-byte groups of K, 8 / MT of them, four to a box; all fragments
        // of up to four groups first, then their conversions and MMAs.
        constexpr int kGroups = 8 / MT, kAhead = NT <= 2 ? (kGroups < 4 ? kGroups : 4) : 1;
#pragma unroll
        for (int k0 = 0; k0 < kGroups; k0 += kAhead) {
          const int group = warp * kGroups + k0;
          if (b0 + (group >> 2) < boxes) {
            uint32_t w8[kAhead][MT][4], x[kAhead][NT][4];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
              const int box = (group + k) >> 2, c = (group + k) & 3;
#pragma unroll
              for (int m = 0; m < MT; ++m)   // 16-byte piece c of a row lies at piece c ^ (row & 7)
                ldmatrix_x4(w8[k][m], stage + box * RU * 128 + m * 16 * 128 + ((c * 32 + a_piece) ^ a_xor));
#pragma unroll
              for (int j = 0; j < NT; ++j)
                if (j < nt) ldmatrix_x4(x[k][j], b_row + j * 8 * L.pitch + (b0 + box) * 256 + c * 64);
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
#pragma unroll
              for (int m = 0; m < MT; ++m) {   // 32 values of K: two MMAs an n-tile
                uint32_t a0[4], a1[4];
                e4m3x4_to_f16(w8[k][m][0], a0[0], a0[2]);
                e4m3x4_to_f16(w8[k][m][1], a0[1], a0[3]);
                e4m3x4_to_f16(w8[k][m][2], a1[0], a1[2]);
                e4m3x4_to_f16(w8[k][m][3], a1[1], a1[3]);
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                  if (j < nt) {
                    mma_f16_m16n8k16(acc[m][j][0], a0, x[k][j][0], x[k][j][1]);
                    mma_f16_m16n8k16(acc[m][j][kAcc - 1], a1, x[k][j][2], x[k][j][3]);
                  }
                }
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
      if (!mbar_wait(&pempty[buf], bph ^ 1u, abort_flag)) {
        if (lane == 0) raise_error(0x4u);
        *abort_flag = 1;
      }
      float* dst = part + buf * kPartFloats + warp * MT * nt * 128 + g * 8 + 2 * t4;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          if (j < nt) {
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              v[i] = kAcc == 2 ? __fadd_rn(acc[m][j][0][i], acc[m][j][kAcc - 1][i]) : acc[m][j][0][i];
            *reinterpret_cast<float2*>(dst + (m * nt + j) * 128) = make_float2(v[0], v[1]);
            *reinterpret_cast<float2*>(dst + (m * nt + j) * 128 + 64) = make_float2(v[2], v[3]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&pfull[buf]);
      if (++buf == kBufs) {
        buf = 0;
        bph ^= 1u;
      }
    }
    k3 = k3 == 2 ? 0 : k3 + 1;
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
      mf_add_weighted(a, w, v);
    }
    mf_store_out(residual, out, static_cast<int64_t>(t) * N + c, a);
  }
}

}  // namespace fp8q
