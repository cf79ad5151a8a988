// Pieces shared by the single-CTA and CTA-pair FP8 GEMM kernels: problem
// parameters, warp roles and the fused dequantization epilogue.
//
// Epilogue arithmetic ("Quantized Inference for OneRec-V2", 关键证据 steps
// 3-4; "FP8量化在生成式推荐系统OneRec-V2中的优化实践" §2.3): the FP32
// accumulator of output (m, n) is scaled by the per-token scale s_x[m] and the
// per-channel scale s_w[n], in that order, each an fp32 multiply rounded to
// nearest, and cast once to fp16 (round to nearest even).
#pragma once

#include <cuda.h>

#include "activation.cuh"
#include "ptx.cuh"

namespace fp8q {

constexpr int kBM = 128;          // rows of a CTA's output slab (TMEM lanes)
constexpr int kBK = 128;          // K bytes per pipeline stage (one 128-B swizzle row)
constexpr int kUmmaK = 32;        // K per tcgen05.mma for 8-bit operands
constexpr int kEpiWarp0 = 2;      // warps 0, 1: TMA producer, MMA issuer
constexpr int kEpiWarps = 8;      // two epilogue warps per TMEM lane quadrant
constexpr int kGemmThreads = (kEpiWarp0 + kEpiWarps) * 32;
// With bias, activation and residual in the epilogue (kEpi): four warps per TMEM
// lane quadrant, one staging tile each.
constexpr int kEpiWarpsFull = 16;
constexpr int epi_warps(bool epi) { return epi ? kEpiWarpsFull : kEpiWarps; }
constexpr int gemm_threads(bool epi) { return (kEpiWarp0 + epi_warps(epi)) * 32; }
constexpr int kStageTileBytes = 32 * 32 * 2;   // one 32 x 32 fp16 output tile per epilogue warp
// Staging for kBufs tiles per epilogue warp: buffer b of warp w at
// (b * kEpiWarps + w) * kStageTileBytes.
__host__ __device__ constexpr int epi_smem_bytes(int bufs) { return bufs * kEpiWarps * kStageTileBytes; }
constexpr int kMaxExperts = 1024;

struct GemmParams {
  const float* s_x;         // [rows]
  const float* s_w;         // [E*N]
  __half* Y;                // [rows, N]
  const int32_t* offsets;   // [E+1] device, grouped only
  const __half* x_f16;      // [rows, K] fp16 activations, fused quantize + GEMM only
  int rows;                 // M (dense) or total grouped rows
  int N;
  int K;
  int E;                    // 1 for dense
  int n_fastest;            // dense tile order: 1 = walk n-blocks first
  // CTA-pair kernel tail split: the first main_tiles full tiles run at full
  // width; each remaining full tile is cut along N into tail_q pieces
  // (tail_q in {1, 2, 4}) so that the last round keeps every cluster busy.
  int main_tiles;
  int tail_q;
  int l2_prefetch;          // split-K: 1 = prefetch the rest of the weight slice into L2 at start
  int half_tiles;           // CTA-pair grouped kernel: an expert's last <= 128 rows as an M = 128 pair tile
  int x_fmt;                // activation code format (Fp8Fmt): E4M3, or E5M2 for the variant
  const uint8_t* xq;        // grouped gather: the token matrix of activation codes [tokens, K]
  const int32_t* row_token; // grouped gather: row r of the product reads token row_token[r] (nullptr: row r)
  int tokens;               // grouped gather / combine: rows of the token matrix
  const int32_t* comb_token; // combine: grouped row r adds into output row comb_token[r] (nullptr: plain store)
  const float* comb_weight;  // combine: the weight of grouped row r
  // CTA-pair dense kernel with the activation quantization inside it: the
  // codes and scales of x_f16 are written to q_out / s_out (= the A operand
  // and s_x); sync holds the per-128-row-block ready flags.
  uint8_t* q_out;
  float* s_out;
  uint32_t* sync;
  // Dense linear with an epilogue (the kEpi kernels):
  // y = fp16(act(acc * s_x * s_w + bias) + residual).
  const __half* bias;       // [N] (nullptr: none)
  const __half* residual;   // [rows, N] (nullptr: none); may be Y itself
  int act;                  // Activation
};

// Row of the activation codes / scales that product row r reads (the row
// itself, or its token in the gathered MoE form; an index out of range reads
// row 0 and is reported by the producer).
__device__ __forceinline__ int act_row(const GemmParams& p, int r) {
  if (p.row_token == nullptr) return r;
  const int t = __ldg(p.row_token + r);
  return (t >= 0 && t < p.tokens) ? t : 0;
}

// One output slab of a CTA: 128 rows starting at row0, BN columns at n0.
struct EpiTile {
  int row0;
  int row_end;   // rows >= row_end are not stored
  int n0;
  int sw0;       // index into s_w of column n0
  bool clip;     // rows >= row_end lie past the output tensor, where a bulk store clips them
};

// Staging layout of a 32 x 32 fp16 tile: row r occupies 64 bytes, its four
// 16-byte chunks permuted as chunk c -> c ^ ((r >> 1) & 3).  This is the
// layout a 64-byte-swizzled TMA box of 32 x 32 fp16 expects (chunk bits 4-5
// XOR address bits 7-8), and it makes both the per-row writes and the
// row-group reads of a warp free of bank conflicts.
__device__ __forceinline__ uint32_t stage_off(int r, int c) {
  return static_cast<uint32_t>(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

// What one epilogue warp drains: 32 output rows from qrow0, nch chunks of
// 32 columns from column col0 of the tile, held in the warp's TMEM lane
// quadrant (q = warp % 4, as tcgen05.ld requires) from TMEM column tcol0.
// Normal tiles: quadrant q holds rows q*32.. of the CTA's 128-row slab and
// the two warps of a quadrant split the bn columns.  Half tiles (a CTA-pair
// MMA with M = 128: 64 rows per CTA) keep the slab's 64 rows twice: lanes
// 0-63 hold columns 0..bn/2-1 and lanes 64-127 columns bn/2..bn-1, both at
// TMEM columns 0..bn/2-1 (measured on B200 with a layout probe).
struct EpiWarpView {
  int qrow0;
  int col0;
  int tcol0;
  int nch;
};

__device__ __forceinline__ EpiWarpView epi_view(const EpiTile& t, int warp, int bn, bool half) {
  const int q = warp & 3;
  const int h = (warp - kEpiWarp0) >> 2;
  EpiWarpView v;
  if (!half) {
    v.qrow0 = t.row0 + q * 32;
    v.col0 = h * (bn / 2);
    v.tcol0 = h * (bn / 2);
    v.nch = bn / 64;
  } else {
    v.qrow0 = t.row0 + (q & 1) * 32;
    v.col0 = (q >> 1) * (bn / 2) + h * (bn / 4);
    v.tcol0 = h * (bn / 4);
    v.nch = bn / 128;
  }
  return v;
}

// The scales one epilogue lane applies: s_x of its row and, for each 32-column
// chunk of its warp, s_w of column (chunk start + lane).  Loaded before the
// wait for the accumulator, so their latency hides behind the tile's MMAs.
template <int kMaxChunks>
struct EpiScales {
  float sx;
  float sw[kMaxChunks];
  float rw;    // combine: weight of this lane's row
  int ctok;    // combine: output (token) row of this lane's row, -1: none
};

template <int kMaxChunks>
__device__ __forceinline__ EpiScales<kMaxChunks> epilogue_scales(const EpiTile& t, const GemmParams& p,
                                                                 const EpiWarpView& w, int lane) {
  EpiScales<kMaxChunks> e;
  const int r = w.qrow0 + lane;
  // With the quantization inside the GEMM (q_out set) s_x is still being
  // written by this kernel: the caller reads it after its block's acquire.
  e.sx = (p.q_out == nullptr && r < t.row_end) ? __ldg(p.s_x + act_row(p, r)) : 0.0f;
  e.rw = 0.0f;
  e.ctok = -1;
  if (p.comb_token != nullptr && r < t.row_end) {
    const int tk = __ldg(p.comb_token + r);
    if (tk >= 0 && tk < p.tokens) {
      e.ctok = tk;
      e.rw = __ldg(p.comb_weight + r);
    } else {
      raise_error(0x8u);
    }
  }
#pragma unroll
  for (int j = 0; j < kMaxChunks; ++j) {
    const int cl = w.col0 + j * 32 + lane;
    e.sw[j] = (j < w.nch && t.n0 + cl < p.N) ? __ldg(p.s_w + t.sw0 + cl) : 0.0f;
  }
  return e;
}

// The epilogue of the dense linear with bias, activation and residual, on the
// 32 columns of one chunk that a lane holds: z = (acc * s_x) * s_w as the
// plain linear computes it, then z + bias, the activation, + residual, each
// fp32 and rounded to nearest; one rounding to fp16.
//
// What it needs besides the accumulators:
//   * s_w and the bias of the tile's columns, which the epilogue warps stage in
//     shared memory while the tile's MMAs run, and all lanes read at the
//     same address (one 16-byte read for four scales or eight biases, where handing
//     them round by shuffles takes an instruction a column);
//   * the residual of the chunk's 32 x 32 values, loaded a chunk ahead four lanes to
//     a row (whole sectors) and turned into rows through the staging tile, which is
//     free then.
constexpr int kEpiColBytes = 256 * (4 + 2);   // s_w fp32, bias fp16 of up to 256 columns (512-wide tiles have no kEpi form)
struct EpiCols {
  float* w;     // [256]
  __half* b;    // [256]
};
__device__ __forceinline__ EpiCols epi_cols(void* after_bars) {
  EpiCols c;
  c.w = reinterpret_cast<float*>((reinterpret_cast<uintptr_t>(after_bars) + 15) & ~uintptr_t(15));
  c.b = reinterpret_cast<__half*>(c.w + 256);
  return c;
}

// What a kEpi epilogue warp does next: its rows of the tile and the values that
// it loads while the tile before is drained, so that no load's latency stands
// between two tiles.
struct EpiNext {
  int n0, bn;        // the tile's columns
  int row0, valid;   // first row of the warp's TMEM lane quadrant, rows that are stored
  float sx;          // scale of the lane's row
  float w;           // scale and bias of column threadIdx.x of the epilogue threads
  __half b;
};
// slab0: first of the CTA's 128 rows.
__device__ __forceinline__ EpiNext epilogue_next(const GemmParams& p, int n0, int bn, int slab0, int row_end) {
  const int tid = threadIdx.x - kEpiWarp0 * 32, lane = tid & 31;
  EpiNext e;
  e.n0 = n0;
  e.bn = bn;
  e.row0 = slab0 + ((threadIdx.x >> 5) & 3) * 32;
  e.valid = row_end - e.row0;
  e.sx = lane < e.valid ? __ldg(p.s_x + e.row0 + lane) : 0.0f;
  const bool in = tid < bn && n0 + tid < p.N;
  e.w = in ? __ldg(p.s_w + n0 + tid) : 0.0f;
  e.b = in && p.bias != nullptr ? __ldg(p.bias + n0 + tid) : __float2half_rn(0.0f);
  // The tile's residual to L2 (128 rows x 512 bytes, a 128-byte line a thread): a
  // chunk's loads are issued one chunk ahead, which covers L2's latency and not HBM's.
  const int r = tid >> 2, c = (tid & 3) * 64;
  if (p.residual != nullptr && c < bn && n0 + c < p.N && slab0 + r < row_end)
    prefetch_l2(p.residual + static_cast<int64_t>(slab0 + r) * p.N + n0 + c);
  return e;
}

// Stage a tile's columns: all kEpi epilogue threads (named barrier 2), before they
// wait for the accumulator; the first barrier ends their reads of the tile before.
__device__ __forceinline__ void epilogue_stage_columns(const EpiCols& c, const EpiNext& e, int tid) {
  named_barrier(2, kEpiWarpsFull * 32);
  if (tid < e.bn) {
    c.w[tid] = e.w;
    c.b[tid] = e.b;
  }
  named_barrier(2, kEpiWarpsFull * 32);
}

// Residual of a chunk (32 rows from row0, 32 columns from n), four lanes to a row:
// r[it] holds columns 8 (lane & 3) .. + 7 of row 8 it + lane / 4.
__device__ __forceinline__ void epilogue_residual(uint4 (&r)[4], const GemmParams& p, int row0, int rows, int n, int lane) {
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    const int row = it * 8 + (lane >> 2), col = n + (lane & 3) * 8;
    r[it] = make_uint4(0, 0, 0, 0);
    if (row < rows && col < p.N) r[it] = ld_global_v4(p.residual + static_cast<int64_t>(row0 + row) * p.N + col);
  }
}

template <int ACT, int P>
__device__ __forceinline__ void activate_pairs(F32x2 (&z)[P]) {
#pragma unroll
  for (int i = 0; i < P; ++i) z[i] = activate2<ACT>(z[i]);
}

template <int P>
__device__ __forceinline__ void activate_pairs_any(F32x2 (&z)[P], int act) {
  switch (act) {   // uniform
    case kActRelu: activate_pairs<kActRelu>(z); break;
    case kActGelu: activate_pairs<kActGelu>(z); break;
    case kActGeluTanh: activate_pairs<kActGeluTanh>(z); break;
    case kActSilu: activate_pairs<kActSilu>(z); break;
    default: break;
  }
}

// One kEpi epilogue warp drains its share of a tile of bn columns: rows of its TMEM
// lane quadrant (warp % 4), 32-column chunks h, h + 4, .. for its h of four (bn / 32
// chunks, two to eight).  `cols`: the tile's staged columns; `res`: the residual of
// the warp's first chunk, and on return of its first chunk of the tile `next`
// (every value of the residual is read by the warp that stores the output in its place,
// before it does, so the residual may be Y itself).
// What bounds it is issue latency, so there are four warps a scheduler, a chunk
// goes through in two halves of 16 columns to fit their registers, and the chunk and
// half loops stay rolled: unrolled like the plain slab the code ran out of the
// instruction cache.  4096 x 8192 x 1024 with bias and GELU, where the epilogue is
// longer than the mainloop: 63 us unrolled, 55 rolled (eight warps, whole chunks).
__device__ __forceinline__ void epilogue_slab_epi(const GemmParams& p, const CUtensorMap* tmY, uint32_t tmem_acc,
                                                  const EpiNext& t, const EpiNext& next, int warp, int lane,
                                                  uint8_t* stage, const EpiCols& cols, uint4 (&res)[4]) {
  const int h32 = ((warp - kEpiWarp0) >> 2) * 32;   // first column of the warp's first chunk
  const uint32_t taddr = tmem_acc + (static_cast<uint32_t>((warp & 3) * 32) << 16);
  const F32x2 sx2 = both(t.sx);
  const uint32_t sbase = smem_u32(stage);
#pragma unroll 1
  for (int cl = h32; cl < t.bn && t.valid > 0; cl += 128) {   // first column of the chunk
    uint32_t v[32];
    tmem_ld_32x32b_x32(taddr + static_cast<uint32_t>(cl), v);
    if (lane == 0) bulk_wait_read_all();   // the staging tile has been read by its last bulk store
    __syncwarp();
    if (p.residual != nullptr) {
#pragma unroll
      for (int it = 0; it < 4; ++it)
        st_shared_v4(sbase + stage_off(it * 8 + (lane >> 2), lane & 3), res[it].x, res[it].y, res[it].z, res[it].w);
      __syncwarp();
      if (cl + 128 < t.bn) epilogue_residual(res, p, t.row0, t.valid, t.n0 + cl + 128, lane);
      else if (h32 < next.bn) epilogue_residual(res, p, next.row0, next.valid, next.n0 + h32, lane);
    }
    tmem_ld_wait_regs(v);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      F32x2 z[8];
      const float* w = cols.w + cl + 16 * h;
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float4 s = *reinterpret_cast<const float4*>(w + 2 * i);
        const uint32_t* a = v + 16 * h + 2 * i;
        z[i] = mul2(mul2(pack2(__uint_as_float(a[0]), __uint_as_float(a[1])), sx2), pack2(s.x, s.y));
        z[i + 1] = mul2(mul2(pack2(__uint_as_float(a[2]), __uint_as_float(a[3])), sx2), pack2(s.z, s.w));
      }
      if (p.bias != nullptr) {   // uniform, as the branches below
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          const uint4 b = *reinterpret_cast<const uint4*>(cols.b + cl + 16 * h + 2 * i);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = __half22float2(reinterpret_cast<const __half2*>(&b)[k]);
            z[i + k] = add2(z[i + k], pack2(f.x, f.y));
          }
        }
      }
      activate_pairs_any(z, p.act);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint32_t at = sbase + stage_off(lane, 2 * h + c);
        if (p.residual != nullptr) {
          const uint4 r = ld_shared_v4(at);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = __half22float2(reinterpret_cast<const __half2*>(&r)[k]);
            z[4 * c + k] = add2(z[4 * c + k], pack2(f.x, f.y));
          }
        }
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float a, b;
          unpack2(z[4 * c + k], a, b);
          const __half2 hv = __floats2half2_rn(a, b);
          o[k] = *reinterpret_cast<const uint32_t*>(&hv);
        }
        st_shared_v4(at, o[0], o[1], o[2], o[3]);
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_2d(tmY, stage, t.n0 + cl, t.row0);   // dense: rows past the end lie past the tensor
      bulk_commit_group();
    }
  }
  // a warp that had nothing to drain in this tile
  if (p.residual != nullptr && (t.valid <= 0 || h32 >= t.bn) && h32 < next.bn)
    epilogue_residual(res, p, next.row0, next.valid, next.n0 + h32, lane);
}

// One epilogue warp drains its view (above), 32 columns at a time:
// TMEM -> registers -> scale and cast -> swizzled staging tile in shared
// memory -> one bulk tensor store.  A warp whose 32 rows all lie past row_end
// does nothing; one whose rows straddle row_end inside the tensor (an MoE
// expert boundary) stores its valid rows with coalesced masked stores
// instead of the bulk store.
// The scales `pre` were loaded before the accumulator wait, the TMEM load of
// chunk j+1 is in flight while chunk j is scaled and stored, and with two
// staging tiles per warp (kBufs = 2) chunk j+1 is written while the bulk
// store of chunk j still reads its tile.  (A slower variant that fetched the
// scales per chunk and waited out every load and store measured no faster
// on the dense shapes and up to 12% slower on the MoE kernels.)
// w.nch <= kMaxChunks.
template <int kMaxChunks, int kBufs>
__device__ __forceinline__ void epilogue_slab(const EpiTile& t, const GemmParams& p, const CUtensorMap* tmY,
                                              uint32_t tmem_acc, const EpiWarpView& w, int warp, int lane,
                                              uint8_t* stage, const EpiScales<kMaxChunks>& pre) {
  static_assert(kBufs == 1 || kBufs == 2, "staging buffers");
  const int q = warp & 3;
  const int nch = w.nch;
  const int qrow0 = w.qrow0;
  const int valid = t.row_end - qrow0;   // rows of this warp that are stored (<= 0: none)
  if (valid <= 0) return;
  // MoE combine: rows go back to their tokens with fp16 atomic adds, read
  // from the staging tile four lanes to a row so that each instruction adds
  // whole 32-byte sectors (half as many L2 atomic operations as one lane per
  // row, 16 bytes at a time).
  const bool combine = p.comb_token != nullptr;
  const bool bulk = !combine && (t.clip || valid >= 32);
  const uint32_t taddr0 = tmem_acc + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(w.tcol0);
  uint32_t v[2][32];
  tmem_ld_32x32b_x32(taddr0, v[0]);
  // Buffer j & 1 below assumes no store of an earlier slab still reads
  // either tile (that slab's last store was issued a whole mainloop ago).
  if (kBufs == 2 && lane == 0) bulk_wait_read_all();
  tmem_ld_wait_regs(v[0]);
#pragma unroll
  for (int j = 0; j < kMaxChunks; ++j) {
    if (j >= nch) break;
    const int cl = w.col0 + j * 32;   // first column of the chunk within the tile
    const uint32_t* cur = v[j & 1];
    if (j + 1 < nch) tmem_ld_32x32b_x32(taddr0 + static_cast<uint32_t>((j + 1) * 32), v[(j + 1) & 1]);
    uint32_t packed[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float w0 = __shfl_sync(0xffffffffu, pre.sw[j], 2 * i);
      const float w1 = __shfl_sync(0xffffffffu, pre.sw[j], 2 * i + 1);
      float y0 = __fmul_rn(__fmul_rn(__uint_as_float(cur[2 * i]), pre.sx), w0);
      float y1 = __fmul_rn(__fmul_rn(__uint_as_float(cur[2 * i + 1]), pre.sx), w1);
      if (combine) {
        y0 = __fmul_rn(y0, pre.rw);
        y1 = __fmul_rn(y1, pre.rw);
      }
      const __half2 hv = __floats2half2_rn(y0, y1);
      packed[i] = *reinterpret_cast<const uint32_t*>(&hv);
    }
    // The staging tile about to be written must have been read by its last
    // bulk store (with two tiles: the store of chunk j-2).
    uint8_t* buf = stage + (kBufs == 2 ? (j & 1) * kEpiWarps * kStageTileBytes : 0);
    if (lane == 0) {
      if (kBufs == 2) bulk_wait_read_1();
      else bulk_wait_read_all();
    }
    __syncwarp();
    const uint32_t sbase = smem_u32(buf);
#pragma unroll
    for (int c = 0; c < 4; ++c)
      st_shared_v4(sbase + stage_off(lane, c), packed[4 * c], packed[4 * c + 1], packed[4 * c + 2], packed[4 * c + 3]);
    if (bulk) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tma_store_2d(tmY, buf, t.n0 + cl, qrow0);
        bulk_commit_group();
      }
    } else {
      __syncwarp();
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const int rr = it * 8 + (lane >> 2);
        const int c = lane & 3;
        const uint4 val = ld_shared_v4(sbase + stage_off(rr, c));
        const int gcol = t.n0 + cl + c * 8;
        if (combine) {
          const int tok = __shfl_sync(0xffffffffu, pre.ctok, rr);   // -1: past the group or rejected
          if (tok >= 0 && gcol < p.N) red_add_f16x8(p.Y + static_cast<int64_t>(tok) * p.N + gcol, val.x, val.y, val.z, val.w);
        } else if (rr < valid && gcol < p.N) {
          *reinterpret_cast<uint4*>(p.Y + static_cast<int64_t>(qrow0 + rr) * p.N + gcol) = val;
        }
      }
      __syncwarp();
    }
    if (j + 1 < nch) tmem_ld_wait_regs(v[(j + 1) & 1]);
  }
}

}  // namespace fp8q
