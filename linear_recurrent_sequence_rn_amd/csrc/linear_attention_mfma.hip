// Linear attention with a decay per head and token over prompts, bf16 in and out, on matrix
// cores. Per head, with c_t the running sum of the log2 decays inside a chunk of 64 tokens and
// S the state in front of it,
//     O = (Q K^T o D) V + diag(2^c) Q S,     D_ts = 2^(c_t - c_s) for s <= t, else 0
//     S <- 2^(c_63) S + K^T (w o V),         w_s = 2^(c_63 - c_s).
//
// A block of four waves owns one segment of one sequence and 4 CW columns of one head's state
// and output; it walks over the segment's chunks with the state in its registers. A wave owns
// CW columns for all rows, so the state never leaves the wave: as accumulator of K^T (w V) it
// has the column in the lane and four rows in the registers, which is just the operand
// layout that Q S needs for its transposed result O^T (rows and columns of the reduction may
// be numbered alike in any order, and all operands here use the order 4g..4g+3,
// 16+4g..16+4g+3 of each 32). K^T and V^T come out of row-major LDS tiles by transposing reads.
// The scores are the one product the waves share: each forms the scores of 16 queries, and
// the tile goes through LDS.
//
// Rounding: the scores times their decay, and the copy of the state that Q S reads, are rounded
// to bf16 once (the outputs are bf16 themselves). The state is float32: w o V is split in
// three bf16 parts, which hold all 24 bits of it, and K is bf16 already, so that the products
// carry float32 accuracy (two parts where only outputs, not the final state, depend on it).
#include "linear_attention.h"

namespace rn {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int kChunk = 64;
constexpr int kThreads = 256;
constexpr double kLog2e = 1.4426950408889634;
constexpr double kFloor = -173.0;      // 2^-173 is 0 in float32: log decays below stand for 0

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Byte offset of element (row, col) in an LDS tile with rows of W bf16. The 16-byte pieces of
// a row are permuted by the row's number, so that both ways of reading are free of bank
// conflicts: 16 rows at one column (operands along the row), and 8 rows times 32 bytes
// (transposing reads).
template <int W>
__device__ __forceinline__ int at(int row, int col) {
  const int f = W == 64 ? (((row >> 1) & 3) << 1 | ((row >> 3) & 1)) : ((row & 7) << 1 | ((row >> 3) & 1));
  return row * (2 * W) + (((col >> 3) ^ f) << 4) + (col & 7) * 2;
}

// Operand whose lane holds row `row`, columns c..c+3 and c+16..c+19 (c = 32 ks + 4 g).
template <int W>
__device__ __forceinline__ bf16x8 row_operand(const char* tile, int row, int c) {
  const uint2 lo = *reinterpret_cast<const uint2*>(tile + at<W>(row, c));
  const uint2 hi = *reinterpret_cast<const uint2*>(tile + at<W>(row, c + 16));
  return __builtin_bit_cast(bf16x8, make_uint4(lo.x, lo.y, hi.x, hi.y));
}
// Operand whose lane holds column col0 + l16, rows r..r+3 and r+16..r+19 (r = 32 ks + 4 g).
template <int W>
__device__ __forceinline__ bf16x8 col_operand(const char* tile, int r, int col0, int l16) {
  const int row = r + (l16 >> 2), col = col0 + (l16 & 3) * 4;
  struct { s16x4 lo, hi; } v;
  v.lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(tile + at<W>(row, col)));
  v.hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(tile + at<W>(row + 16, col)));
  return __builtin_bit_cast(bf16x8, v);
}

struct alignas(16) Decays {   // of one chunk
  float c[kChunk];       // running sum of log2 decays
  float e[kChunk];       // 2^c
  float w[kChunk];       // 2^(c_63 - c)
  float a;               // 2^c_63
  int bad;               // v holds a NaN or an infinity
};

// Wave 0: the decays of a chunk from each lane's log decay. Sums in float64, so that
// differences of far sums keep float32 accuracy. Returns the chunk's sum of log2 decays.
__device__ __forceinline__ double scan_decays(float g, Decays* d) {
  const int lane = threadIdx.x & 63;
  double x = static_cast<double>(g) * kLog2e;
  if (x < kFloor) x = kFloor;           // (a NaN stays)
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const double y = __shfl_up(x, o, 64);
    if (lane >= o) x += y;
  }
  const double last = __shfl(x, 63, 64);
  d->c[lane] = static_cast<float>(x);
  d->e[lane] = exp2f(static_cast<float>(x));
  d->w[lane] = exp2f(static_cast<float>(last - x));
  if (lane == 63) d->a = exp2f(static_cast<float>(x));
  return last;
}

// One 64-row tile of W columns on its way from memory to LDS: 16 bytes a thread and step.
template <int W>
struct Tile {
  static constexpr int kPer = W / 8;                       // 16-byte pieces a row
  static constexpr int kStep = kThreads / kPer;            // rows a step
  static constexpr int kN = kChunk / kStep;
  uint4 r[kN];
  // Rows t0.. of `p` (row stride st, `cols` columns in use); rows past `last` read row `last`.
  __device__ __forceinline__ void load(const uint16_t* p, int64_t st, int t0, int last, int cols) {
    const int row = threadIdx.x / kPer, c = threadIdx.x % kPer * 8;
    const uint16_t* q = p + (c < cols ? c : 0);
#pragma unroll
    for (int i = 0; i < kN; ++i)
      r[i] = *reinterpret_cast<const uint4*>(q + min(t0 + row + i * kStep, last) * st);
  }
  // Into LDS; rows from `rows` on and columns from `cols` on become zeros.
  __device__ __forceinline__ void store(char* tile, int rows, int cols) {
    const int row = threadIdx.x / kPer, c = threadIdx.x % kPer * 8;
    const bool whole = rows >= kChunk && cols >= W;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      if (!whole && (c >= cols || row + i * kStep >= rows)) r[i] = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(tile + at<W>(row + i * kStep, c)) = r[i];
    }
  }
  // Whether a value is a NaN or an infinity (largest exponent).
  __device__ __forceinline__ bool nonfinite() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const uint32_t u[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t hi = (u[j] & 0x7fff0000u), lo = (u[j] & 0x7fffu) << 16;
        m = max(m, max(hi, lo));
      }
    }
    return m >= 0x7f800000u;
  }
};

template <int DK, int CW, LinMode MODE>
__global__ void __launch_bounds__(kThreads, DK == 256 ? 1 : 2) lin_chunks(LinArgs a, int slices) {
  constexpr int DV = 4 * CW;             // columns a block
  constexpr int VT = CW / 16;            // 16-column tiles a wave
  constexpr int AT = DK / 16;            // 16-row tiles of the state
  constexpr int KS = DK / 32;            // reduction steps along d_k
  constexpr int PARTS = MODE == kLinOut ? 2 : 3;
  constexpr bool kOut = MODE != kLinState;
  __shared__ __align__(16) char smem[(kOut ? 2 : 1) * kChunk * DK * 2 + kChunk * DV * 2 + (kOut ? kChunk * kChunk * 2 : 0)];
  __shared__ __align__(16) Decays dec[2];
  char* kt = smem;
  char* vt = kt + kChunk * DK * 2;
  char* qt = vt + kChunk * DV * 2;
  char* pt = qt + kChunk * DK * 2;

  const int h = blockIdx.x / slices, c0 = (blockIdx.x - h * slices) * DV;
  const int seg = blockIdx.y, s = blockIdx.z;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l16 = lane & 15, g4 = (lane >> 4) * 4;
  const int nc = min(DV, a.dv - c0);
  int64_t row0, own;
  int len;
  lin_span(a, s, &row0, &len, &own);
  if (kOut && a.zero_rest) lin_zero_rest<RN_BF16>(a, s, seg, h, c0, nc, row0, len, own);
  if (s == a.S) return;
  const int t0 = seg * a.seg_len, t1 = min(len, t0 + a.seg_len);
  const int slot = lin_slot(a, s);
  const bool keep = a.state_out && slot >= 0;
  if (MODE == kLinWhole ? (len == 0 && !keep) : t0 >= t1) return;
  if (MODE == kLinState && t1 == len && !keep) return;   // nobody reads the last segment's state

  const int64_t sh = static_cast<int64_t>(a.dk) * a.dv;
  const int vcol = c0 + wave * CW + l16;                 // this lane's state columns: vcol + 16 j
  f32x4 S[AT][VT];
  {
    const float* from = MODE == kLinWhole ? (a.state_in && slot >= 0 ? a.state_in + (static_cast<int64_t>(slot) * a.H + h) * sh : nullptr)
                        : MODE == kLinOut ? a.seg_state + (lin_segment(a, s, row0, seg) * a.H + h) * sh
                                          : nullptr;
#pragma unroll
    for (int i = 0; i < AT; ++i)
#pragma unroll
      for (int j = 0; j < VT; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int d = 16 * i + g4 + r, v = vcol + 16 * j;
          S[i][j][r] = from && d < a.dk && v < a.dv ? from[static_cast<int64_t>(d) * a.dv + v] : 0.f;
        }
  }
  const uint16_t* qp = static_cast<const uint16_t*>(a.q) + lin_base(a, a.qs, s, row0) + h / (a.H / a.Hq) * a.qs[1];
  const uint16_t* kp = static_cast<const uint16_t*>(a.k) + lin_base(a, a.ks, s, row0) + h / (a.H / a.Hk) * a.ks[1];
  const uint16_t* vp = static_cast<const uint16_t*>(a.v) + lin_base(a, a.vs, s, row0) + h / (a.H / a.Hv) * a.vs[1] + c0;
  const float* gp = a.g + lin_base(a, a.gs, s, row0) + h * a.gs[1];
  uint16_t* op = static_cast<uint16_t*>(a.out) + lin_base(a, a.os, s, row0) + h * a.os[1] + c0 + wave * CW;

  Tile<DK> tq, tk;
  Tile<DV> tv;
  auto fetch = [&](int t) {
    if constexpr (kOut) tq.load(qp, a.qs[2], t, len - 1, a.dk);
    tk.load(kp, a.ks[2], t, len - 1, a.dk);
    tv.load(vp, a.vs[2], t, len - 1, nc);
  };
  auto log_decay = [&](int t) { return t + lane < t1 ? gp[(t + lane) * a.gs[2]] : 0.f; };

  double gsum = 0.0;
  float gnext = 0.f;
  if (t0 < t1) {
    fetch(t0);
    if (wave == 0) {
      gsum += scan_decays(log_decay(t0), &dec[0]);
      gnext = log_decay(t0 + kChunk);
    }
    if (tid == 0) dec[0].bad = 0;
    if constexpr (kOut) {   // score tiles above the diagonal that the products read
      for (int i = tid; i < 2 * 16 * 4; i += kThreads) {
        const int t = (i >> 6) * 32 + (i & 15), col = (i >> 6) * 32 + 16 + ((i >> 4) & 3) * 4;
        *reinterpret_cast<uint2*>(pt + at<kChunk>(t, col)) = make_uint2(0, 0);
      }
    }
    __syncthreads();
  }
  int buf = 0;
  for (int t = t0; t < t1; t += kChunk, buf ^= 1) {
    const int n = min(kChunk, t1 - t);
    if (tv.nonfinite()) dec[buf].bad = 1;   // (columns past d_v repeat others of the row)
    if constexpr (kOut) tq.store(qt, n, a.dk);
    tk.store(kt, n, a.dk);
    tv.store(vt, n, nc);
    __syncthreads();
    const Decays& D = dec[buf];
    if (t + kChunk < t1) {
      fetch(t + kChunk);
      if (wave == 0) {
        gsum += scan_decays(gnext, &dec[buf ^ 1]);
        gnext = log_decay(t + 2 * kChunk);
      }
      if (tid == 0) dec[buf ^ 1].bad = 0;
    }
    f32x4 O[4][VT];
    if constexpr (kOut) {
      // scores of the 16 queries of this wave: P^T = K Q^T, keys in the rows
      const int tw = 16 * wave + l16;
      const float ct = D.c[tw];
      bf16x8 qf[KS];
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) qf[ks] = row_operand<DK>(qt, tw, 32 * ks + g4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i > wave) break;
        f32x4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) p = mfma(row_operand<DK>(kt, 16 * i + l16, 32 * ks + g4), qf[ks], p);
        const f32x4 cs = *reinterpret_cast<const f32x4*>(&D.c[16 * i + g4]);
        float x[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] = 16 * i + g4 + r <= tw ? p[r] * exp2f(ct - cs[r]) : 0.f;
        *reinterpret_cast<uint2*>(pt + at<kChunk>(tw, 16 * i + g4)) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
      }
      // what the state in front of the chunk gives: O^T = S^T Q^T, scaled by 2^c of the query
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int v = 0; v < VT; ++v) O[j][v] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        bf16x8 sf[VT];
#pragma unroll
        for (int v = 0; v < VT; ++v) {
          const f32x4 x = S[2 * ks][v], y = S[2 * ks + 1][v];
          sf[v] = __builtin_bit_cast(bf16x8, make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                        pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bf16x8 q = row_operand<DK>(qt, 16 * j + l16, 32 * ks + g4);
#pragma unroll
          for (int v = 0; v < VT; ++v) O[j][v] = mfma(sf[v], q, O[j][v]);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float e = D.e[16 * j + l16];
#pragma unroll
        for (int v = 0; v < VT; ++v) O[j][v] *= e;
      }
      __syncthreads();                      // the score tile is whole
    }
    const bool bad = D.bad;
    bf16x8 vf[2][VT];
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int v = 0; v < VT; ++v) vf[ks][v] = col_operand<DV>(vt, 32 * ks + g4, wave * CW + 16 * v, l16);
    if constexpr (kOut) {
      if (!bad) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int ks = 0; ks <= j / 2; ++ks) {
            const bf16x8 p = row_operand<kChunk>(pt, 16 * j + l16, 32 * ks + g4);
#pragma unroll
            for (int v = 0; v < VT; ++v) O[j][v] = mfma(vf[ks][v], p, O[j][v]);
          }
      } else {
        // 0 times a NaN or an infinity of a later token must not reach this one: the same sums,
        // over the tokens up to the query's only
        for (int j = 0; j < 4; ++j)
          for (int k = 0; k < 16 * j + 16; ++k) {
            const int q = 16 * j + l16;
            const float p = bf16_to_f32(*reinterpret_cast<const uint16_t*>(pt + at<kChunk>(q, k)));
#pragma unroll
            for (int v = 0; v < VT; ++v) {
              const uint2 x = *reinterpret_cast<const uint2*>(vt + at<DV>(k, wave * CW + 16 * v + g4));
              const float y[4] = {__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u),
                                  __uint_as_float(x.y << 16), __uint_as_float(x.y & 0xffff0000u)};
#pragma unroll
              for (int jj = 0; jj < 4; ++jj)
                if (jj == j)
#pragma unroll
                  for (int r = 0; r < 4; ++r) O[jj][v][r] = k <= q ? fmaf(p, y[r], O[jj][v][r]) : O[jj][v][r];
            }
          }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int tt = 16 * j + l16;
#pragma unroll
        for (int v = 0; v < VT; ++v) {
          const f32x4 o = O[j][v] * a.scale;
          if (tt < n && wave * CW + 16 * v + g4 < nc)
            *reinterpret_cast<uint2*>(op + (t + tt) * a.os[2] + 16 * v + g4) = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
        }
      }
    }
    if (MODE != kLinOut || t + kChunk < t1) {
      // S <- a S + K^T (w V): the parts of w V in the same order of tokens as K^T
      bf16x8 wf[2][VT][PARTS];
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const f32x4 w0 = *reinterpret_cast<const f32x4*>(&D.w[32 * ks + g4]);
        const f32x4 w1 = *reinterpret_cast<const f32x4*>(&D.w[32 * ks + 16 + g4]);
#pragma unroll
        for (int v = 0; v < VT; ++v) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float x = static_cast<float>(vf[ks][v][j]) * (j < 4 ? w0[j & 3] : w1[j & 3]);
#pragma unroll
            for (int p = 0; p < PARTS; ++p) {
              wf[ks][v][p][j] = static_cast<__bf16>(x);
              x -= static_cast<float>(wf[ks][v][p][j]);
            }
          }
          if (bad)                          // an infinity has no lower parts
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (!(fabsf(static_cast<float>(wf[ks][v][0][j])) < INFINITY))
#pragma unroll
                for (int p = 1; p < PARTS; ++p) wf[ks][v][p][j] = static_cast<__bf16>(0.f);
        }
      }
      const float dec64 = D.a;
#pragma unroll
      for (int i = 0; i < AT; ++i) {
#pragma unroll
        for (int v = 0; v < VT; ++v) S[i][v] *= dec64;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          const bf16x8 kf = col_operand<DK>(kt, 32 * ks + g4, 16 * i, l16);
#pragma unroll
          for (int v = 0; v < VT; ++v)
#pragma unroll
            for (int p = PARTS - 1; p >= 0; --p) S[i][v] = mfma(kf, wf[ks][v][p], S[i][v]);
        }
      }
    }
    __syncthreads();                        // the tiles are free
  }
  float* to = nullptr;
  if (MODE == kLinWhole && keep) to = a.state_out + (static_cast<int64_t>(slot) * a.H + h) * sh;
  if (MODE == kLinState) {
    const int64_t i = lin_segment(a, s, row0, seg) * a.H + h;
    to = a.seg_state + i * sh;
    if (c0 == 0 && tid == 0) a.seg_decay[i] = exp2f(static_cast<float>(gsum));
  }
  if (to) {
#pragma unroll
    for (int i = 0; i < AT; ++i)
#pragma unroll
      for (int j = 0; j < VT; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int d = 16 * i + g4 + r, v = vcol + 16 * j;
          if (d < a.dk && v < a.dv) to[static_cast<int64_t>(d) * a.dv + v] = S[i][j][r];
        }
  }
}

// Columns a wave: 32 where d_v has a second half for them (each chunk's Q and K are then read
// from LDS for twice the columns), else 16.
int columns(const LinArgs& a) { return a.dv > 64 ? 32 : 16; }

template <int DK, int CW>
hipError_t launch_t(const LinArgs& a, LinMode mode, hipStream_t st) {
  const int slices = (a.dv + 4 * CW - 1) / (4 * CW);
  const bool rest = a.T > 0 && a.zero_rest && mode != kLinState;
  const dim3 grid(a.H * slices, a.n_seg, a.S + (rest ? 1 : 0));
  if (mode == kLinWhole) hipLaunchKernelGGL((lin_chunks<DK, CW, kLinWhole>), grid, dim3(kThreads), 0, st, a, slices);
  else if (mode == kLinState) hipLaunchKernelGGL((lin_chunks<DK, CW, kLinState>), grid, dim3(kThreads), 0, st, a, slices);
  else hipLaunchKernelGGL((lin_chunks<DK, CW, kLinOut>), grid, dim3(kThreads), 0, st, a, slices);
  return hipGetLastError();
}

}  // namespace

int lin_mfma_blocks(const LinArgs& a) {
  const int w = 4 * columns(a);
  return a.H * ((a.dv + w - 1) / w);
}

hipError_t launch_lin_mfma(const LinArgs& a, LinMode mode, hipStream_t st) {
  const bool wide = columns(a) == 32;
  if (a.dk <= 64) return wide ? launch_t<64, 32>(a, mode, st) : launch_t<64, 16>(a, mode, st);
  if (a.dk <= 128) return wide ? launch_t<128, 32>(a, mode, st) : launch_t<128, 16>(a, mode, st);
  return wide ? launch_t<256, 32>(a, mode, st) : launch_t<256, 16>(a, mode, st);
}

}  // namespace rn
