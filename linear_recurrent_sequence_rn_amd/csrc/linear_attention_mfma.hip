// Linear attention with a decay per head and token over prompts, bf16 in and out, on matrix
// cores. Per head, with c_t the running sum of the log2 decays inside a chunk of 64 tokens and
// S the state in front of it,
//     O = (Q K^T o D) V + diag(2^c) Q S,     D_ts = 2^(c_t - c_s) for s <= t, else 0
//     S <- 2^(c_63) S + K^T (w o V),         w_s = 2^(c_63 - c_s).
//
// A block owns one segment of one sequence and VW CW columns of one head's state and output;
// it walks over the segment's chunks with the state in its registers. A wave owns CW columns
// and d_k / DW rows, so the state never leaves the wave: as accumulator of K^T (w V) it has
// the column in the lane and four rows in the registers, which is just the operand layout
// that Q S needs for its transposed result O^T (rows and columns of the reduction may be
// numbered alike in any order, and all operands here use the order 4g..4g+3,
// 16+4g..16+4g+3 of each 32). K^T and V^T come out of row-major LDS tiles by transposing reads.
// The scores are shared by all waves: their ten 16 x 16 tiles are dealt out by key tile and meet
// in LDS. With DW = 2 the two waves of a column pair each have a share of Q S of every query;
// each hands the other its share of two of the four query tiles, through LDS.
//
// A chunk takes two barriers: tiles written; scores, Q S and the new state formed (after it only
// the score tile, the shares and registers are read, so the next chunk's tiles may be written).
// The next tiles are on their way in registers meanwhile.
//
// What bounds it: heads of 256 x 512, the matrix cores at the clock they reach under load (8192
// tokens, 16 heads: 350 us for 266 GFLOP, of which the three parts of w V are 103; under the profiler
// states 124 us, scan 13 us, outputs 293 us; one large bf16 product reaches 1230 TFLOP/s on the
// card). Heads of 64 and 128: instruction issue, about 540 vector and 57 matrix instructions a wave
// and chunk at d_k 64, with two or three blocks a CU (13 packed sequences, 14001 tokens, 32 heads of
// 64 x 128: 137 to 185 us, by how long the longest is, 1.6 to 2.1 TB/s; 8 sequences of 2048 tokens, 32
// heads of 128 x 128: 193 us, 2.8 TB/s).
//
// Rounding: Q, K and V are bf16 already, and what is formed from them in float32 enters a product
// in several bf16 parts. Outputs depend on two parts of each score times its decay, of the state's
// copy that Q S reads and, in the pass that only gives outputs, of w o V: what two parts leave out is
// at most 2^-16 of the value, 1/256 of the one rounding that a bf16 output takes (one part, which is
// 45 us less for 8192 tokens of 16 heads of 256 x 512, doubles that rounding). The state that is kept
// is float32: w o V in three parts, which hold all 24 bits of it.
#include <type_traits>

#include "linear_attention.h"

namespace rn {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int kChunk = 64;
constexpr double kLog2e = 1.4426950408889634;
// Log decays below stand for 0: 2^-300 is 0 in float32, also times the largest scale.
constexpr double kFloor = -300.0;

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

// Tiles whose rows are read as row operands have 64 bytes behind each 16 rows: two such reads a
// whole number of 512 bytes apart would become one instruction whose halves meet in the same banks
// (18 cycles in place of 2 x 4; 8 x 2048 tokens, 32 heads of 128 x 128: 193 us, without them 199).
constexpr int kGap = 64;
template <int W>
constexpr int kRows = 32 * W + kGap;    // bytes of 16 rows
template <int W>
__device__ __forceinline__ int at_gap(int row, int col) { return at<W>(row, col) + (row >> 4) * kGap; }

// The permutation only XORs bits of the offset, and so do steps of whole 16 columns: all offsets
// a lane needs come from one base per way of reading, XORed with constants, and from
// constants added for steps of 16 rows.
//
// Operand whose lane holds its row, columns c..c+3 and c+16..c+19 with c = 32 ks + g4;
// base = at<W>(l16, g4), rows = byte offset of the tile of 16 rows.
__device__ __forceinline__ bf16x8 row_operand(const char* tile, int base, int ks, int rows) {
  const uint2 lo = *reinterpret_cast<const uint2*>(tile + (base ^ (ks << 6)) + rows);
  const uint2 hi = *reinterpret_cast<const uint2*>(tile + (base ^ (ks << 6 | 32)) + rows);
  return __builtin_bit_cast(bf16x8, make_uint4(lo.x, lo.y, hi.x, hi.y));
}
// Operand whose lane holds column 16 i + l16, rows r..r+3 and r+16..r+19 with r = 32 ks + g4;
// base = at<W>(g4 + l16 / 4, 4 (l16 % 4)).
template <int ROWS>   // bytes of 16 rows
__device__ __forceinline__ bf16x8 col_operand(const char* tile, int base, int ks, int i) {
  const char* p = tile + (base ^ (i << 5)) + ks * (2 * ROWS);
  struct { s16x4 lo, hi; } v;
  v.lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p));
  v.hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + ROWS));
  return __builtin_bit_cast(bf16x8, v);
}

// Byte offset of a score's lower part, from that of its upper part: queries 0 .. 31 (row tiles 0 and
// 1) see keys 0 .. 31 only, whose lower parts take the columns 32 .. 63 of the same rows; the
// others' are in two more row tiles.
__device__ __forceinline__ int low_part(int p, int tile) {
  const int t0 = tile * kRows<kChunk>;
  return tile < 2 ? ((p - t0) ^ 64) + t0 : p + 2 * kRows<kChunk>;
}

// For the lower parts of values of which the largest is `top`: none where an upper part is an
// infinity (what is left of it would be a NaN; the output that such values reach has no others).
__device__ __forceinline__ uint32_t low_mask(float top) { return top <= 0x1.fep127f ? ~0u : 0u; }

struct alignas(16) Decays {   // of one chunk
  // Running sum of log2 decays, as the sum of two floats: with zeros among the decays it passes 1e4,
  // and differences of such sums keep float32 accuracy only if both parts are subtracted.
  float c[kChunk];
  float l[kChunk];
  float q[kChunk];       // l + log2 |scale|: the queries' side of a score's decay
  float e[kChunk];       // 2^c |scale|
  float w[kChunk];       // 2^(c_63 - c)
  float a;               // 2^c_63
  int bad;               // v holds a NaN or an infinity
};

// x and y in PARTS bf16 parts each, packed in pairs at out[0], out[stride], ...; with SAFE an
// infinity or NaN has no lower parts.
template <int PARTS, bool SAFE>
__device__ __forceinline__ void split_pair(float x, float y, uint32_t* out, int stride) {
#pragma unroll
  for (int p = 0; p < PARTS; ++p) {
    const uint32_t u = pack_bf16x2(x, y);
    out[p * stride] = u;
    if (p + 1 < PARTS) {
      const float hx = __uint_as_float(u << 16), hy = __uint_as_float(u & 0xffff0000u);
      x -= hx;
      y -= hy;
      if (SAFE) {
        if (!(fabsf(hx) < INFINITY)) x = 0.f;
        if (!(fabsf(hy) < INFINITY)) y = 0.f;
      }
    }
  }
}

// x moved across lanes by a DPP control; lanes without a source (or outside the row mask) get 0.
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_or_zero(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(u), CTRL, ROWS, 0xf, true);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(u >> 32), CTRL, ROWS, 0xf, true);
  return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}

// One wave: the decays of a chunk from each lane's log decay, their sums in float64. Returns the
// chunk's sum of log2 decays.
__device__ __forceinline__ double scan_decays(float g, float log2_scale, Decays* d) {
  const int lane = threadIdx.x & 63;
  double x = static_cast<double>(g) * kLog2e;
  if (x < kFloor) x = kFloor;           // (a NaN stays)
  x += dpp_or_zero<0x111, 0xf>(x);      // inclusive sums over the 16 lanes of a row ...
  x += dpp_or_zero<0x112, 0xf>(x);
  x += dpp_or_zero<0x114, 0xf>(x);
  x += dpp_or_zero<0x118, 0xf>(x);
  x += dpp_or_zero<0x142, 0xa>(x);      // ... lane 15 into rows 1 and 3, lane 31 into rows 2 and 3
  x += dpp_or_zero<0x143, 0xc>(x);
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(u), 63);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(u >> 32), 63);
  const double last = __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
  const float c = static_cast<float>(x);
  const float l = static_cast<float>(x - c);
  d->c[lane] = c;
  d->l[lane] = l;
  d->q[lane] = l + log2_scale;
  d->e[lane] = exp2f(static_cast<float>(x + log2_scale));
  d->w[lane] = exp2f(static_cast<float>(last - x));
  if (lane == 63) d->a = exp2f(static_cast<float>(x));
  return last;
}

// One 64-row tile of W columns on its way from memory to LDS: 16 bytes a thread and step.
// The chunk's start is a scalar; offsets inside a chunk are 32 bits where the stride allows it.
template <int W, int NT>
struct Tile {
  static constexpr int kPer = W / 8;                       // 16-byte pieces a row
  static constexpr int kStep = NT / kPer;                  // rows a step
  static constexpr int kN = kChunk / kStep;
  uint4 r[kN];
  // This thread's offset in a chunk whose 64 rows all exist.
  static __device__ __forceinline__ uint32_t lane_offset(int64_t st, int cols) {
    const int row = threadIdx.x / kPer, c = threadIdx.x % kPer * 8;
    return row * static_cast<uint32_t>(st) + (c < cols ? c : 0);
  }
  // The 64 rows from `p` on (row stride st, `cols` columns in use), of which `rows` exist: the
  // others repeat the last one.
  __device__ __forceinline__ void load(const uint16_t* p, int64_t st, uint32_t off, int rows, int cols) {
    if (rows >= kChunk && st < (1 << 24)) {
#pragma unroll
      for (int i = 0; i < kN; ++i) r[i] = *reinterpret_cast<const uint4*>(p + i * kStep * st + off);
    } else {
      const int row = threadIdx.x / kPer, c = threadIdx.x % kPer * 8;
#pragma unroll
      for (int i = 0; i < kN; ++i)
        r[i] = *reinterpret_cast<const uint4*>(p + min(row + i * kStep, rows - 1) * st + (c < cols ? c : 0));
    }
  }
  // Rows from `rows` on and columns from `cols` on become zeros.
  __device__ __forceinline__ void trim(int rows, int cols) {
    if (rows >= kChunk && cols >= W) return;
    const int row = threadIdx.x / kPer, c = threadIdx.x % kPer * 8;
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (c >= cols || row + i * kStep >= rows) r[i] = make_uint4(0, 0, 0, 0);
  }
  template <bool GAP>
  __device__ __forceinline__ void store(char* tile) const {
    const int row = threadIdx.x / kPer, c = threadIdx.x % kPer * 8;
#pragma unroll
    for (int i = 0; i < kN; ++i)
      *reinterpret_cast<uint4*>(tile + (GAP ? at_gap<W>(row + i * kStep, c) : at<W>(row + i * kStep, c))) = r[i];
  }
  // Whether a value is a NaN or an infinity (largest exponent).
  __device__ __forceinline__ bool nonfinite() const {
    typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
    u16x2 m = {0, 0};
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const uint32_t u[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, u[j] & 0x7fff7fffu));
    }
    return max(m.x, m.y) >= 0x7f80;
  }
  // The values of step i times w, in PARTS bf16 parts that add up to it, largest first.
  template <int PARTS, bool SAFE>
  __device__ __forceinline__ void split(int i, float w, uint4* part) const {
    const uint32_t u[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
    uint32_t o[PARTS][4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      split_pair<PARTS, SAFE>(__uint_as_float(u[j] << 16) * w, __uint_as_float(u[j] & 0xffff0000u) * w, &o[0][j], 4);
#pragma unroll
    for (int p = 0; p < PARTS; ++p) part[p] = make_uint4(o[p][0], o[p][1], o[p][2], o[p][3]);
  }
};

template <int DK, int CW, int VW, int DW, LinMode MODE>
__global__ void __launch_bounds__(64 * VW * DW, DK == 64 ? 3 : 2) lin_chunks(LinArgs a) {
  constexpr int NT = 64 * VW * DW;
  constexpr int DV = VW * CW;            // columns a block
  constexpr int VT = CW / 16;            // 16-column tiles a wave
  constexpr int AT = DK / 16 / DW;       // 16-row tiles of the state a wave
  constexpr int KS = DK / 32;            // reduction steps along d_k
  constexpr int OT = 4 / DW;             // 16-query tiles of the output a wave finishes
  constexpr int PARTS = MODE == kLinOut ? 2 : 3;
  constexpr bool kOut = MODE != kLinState;
  // (the scores' upper parts in four row tiles; see low_part() for the lower ones)
  constexpr int kTileQ = 4 * kRows<DK>, kTileV = kChunk * DV * 2, kTileP = 6 * kRows<kChunk>;
  constexpr int kSwap = DW == 2 ? VW * DW * 2 * VT * 1024 : 0;
  // Two waves need each part of w V where DW is 2: they are formed once, on the way to LDS, as
  // long as the tiles fit in it; else each wave forms its own in registers.
  constexpr int kBase = kTileQ + (kOut ? kTileV + kTileQ + kTileP + kSwap : 0);
  constexpr bool kParts = DW == 2 && kBase + PARTS * kTileV + 2 * sizeof(Decays) <= 160 * 1024;
  constexpr bool kHasV = kOut || !kParts;    // V itself is needed in LDS
  __shared__ __align__(16) char smem[kBase + (kParts ? PARTS * kTileV : 0) + (kOut || kParts ? 0 : kTileV)];
  __shared__ Decays dec[2];
  char* kt = smem;
  char* vt = kt + kTileQ;
  char* wt = vt + (kHasV ? kTileV : 0);
  char* qt = wt + (kParts ? PARTS * kTileV : 0);
  char* pt = qt + kTileQ;
  f32x4* swap = reinterpret_cast<f32x4*>(pt + kTileP);

  int h, c0;
  lin_block(a, blockIdx.x, &h, &c0);
  c0 *= DV;
  int seg, s;
  if (!lin_place(a, &s, &seg)) return;
  const int tid = threadIdx.x;
  const int lane = tid & 63, l16 = lane & 15, g4 = (lane >> 4) * 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wv = wave % VW, wd = wave / VW;              // column tile and row half of this wave
  // Key tile of this wave's scores: the first meets four query tiles, the last one, so the tiles
  // go round the waves (and SIMDs) from block to block.
  const int keys = (wave + blockIdx.x) & 3;
  const int nc = min(DV, a.dv - c0);
  int64_t row0, own;
  int len;
  lin_span(a, s, &row0, &len, &own);
  if (kOut && a.zero_rest) lin_zero_rest<RN_BF16>(a, s, seg, h, c0, nc, row0, len, own);
  if (s == a.S) return;
  const int t0 = min(seg, a.n_seg) * a.seg_len, t1 = min(len, t0 + a.seg_len);
  const int slot = lin_slot(a, s);
  const bool keep = a.state_out && slot >= 0;
  const bool one = len <= a.seg_len;      // (always, where kLinWhole is the only pass)
  if (t0 >= t1 && !(MODE == kLinWhole && seg == 0 && keep)) return;
  if (MODE == kLinState && t1 == len && (!keep || (a.flat && one))) return;   // nobody reads the last segment's state

  const int64_t sh = static_cast<int64_t>(a.dk) * a.dv;
  const int vcol = c0 + wv * CW + l16;                   // this lane's state columns: vcol + 16 j
  const int drow = wd * (DK / DW);                       // and rows: drow + 16 i + g4 + r
  f32x4 S[AT][VT];
  {
    const float* from = MODE == kLinState ? nullptr
                        : MODE == kLinOut || !one ? a.seg_state + (lin_segment(a, s, row0, seg) * a.H + h) * sh
                        : a.state_in && slot >= 0 ? a.state_in + (static_cast<int64_t>(slot) * a.H + h) * sh : nullptr;
#pragma unroll
    for (int i = 0; i < AT; ++i)
#pragma unroll
      for (int j = 0; j < VT; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int d = drow + 16 * i + g4 + r, v = vcol + 16 * j;
          S[i][j][r] = from && d < a.dk && v < a.dv ? from[static_cast<int64_t>(d) * a.dv + v] : 0.f;
        }
  }
  const uint16_t* qp = static_cast<const uint16_t*>(a.q) + lin_base(a, a.qs, s, row0) + h / (a.H / a.Hq) * a.qs[1];
  const uint16_t* kp = static_cast<const uint16_t*>(a.k) + lin_base(a, a.ks, s, row0) + h / (a.H / a.Hk) * a.ks[1];
  const uint16_t* vp = static_cast<const uint16_t*>(a.v) + lin_base(a, a.vs, s, row0) + h / (a.H / a.Hv) * a.vs[1] + c0;
  const float* gp = a.g + lin_base(a, a.gs, s, row0) + h * a.gs[1];
  uint16_t* op = static_cast<uint16_t*>(a.out) + lin_base(a, a.os, s, row0) + h * a.os[1] + c0 + wv * CW;

  Tile<DK, NT> tq, tk;
  Tile<DV, NT> tv;
  const uint32_t qoff = tq.lane_offset(a.qs[2], a.dk), koff = tk.lane_offset(a.ks[2], a.dk), voff = tv.lane_offset(a.vs[2], nc);
  auto fetch_q = [&](int t) {
    if constexpr (kOut) tq.load(qp + t * a.qs[2], a.qs[2], qoff, len - t, a.dk);
  };
  auto fetch_k = [&](int t) { tk.load(kp + t * a.ks[2], a.ks[2], koff, len - t, a.dk); };
  auto fetch_v = [&](int t) { tv.load(vp + t * a.vs[2], a.vs[2], voff, len - t, nc); };
  auto log_decay = [&](int t) { return t + lane < t1 ? gp[(t + lane) * a.gs[2]] : 0.f; };

  const float log2_scale = log2f(fabsf(a.scale));   // (-inf for 0: the outputs become 0)
  double gsum = 0.0;
  float gnext = 0.f;
  if (t0 < t1) {
    fetch_v(t0);
    fetch_k(t0);
    fetch_q(t0);
    if (wave == NT / 64 - 1) {              // (the last wave has the fewest score tiles)
      gsum += scan_decays(log_decay(t0), log2_scale, &dec[0]);
      gnext = log_decay(t0 + kChunk);
    }
    if (tid == 0) dec[0].bad = 0;
    if constexpr (kOut) {                   // score tiles above the diagonal that are read
      if (tid < 2 * 16 * 4) {
        const int tt = (tid >> 6) * 32 + (tid & 15), col = (tid >> 6) * 32 + 16 + ((tid >> 4) & 3) * 4;
        const int p = at_gap<kChunk>(tt, col);
        *reinterpret_cast<uint2*>(pt + p) = make_uint2(0, 0);
        *reinterpret_cast<uint2*>(pt + low_part(p, tt >> 4)) = make_uint2(0, 0);
      }
    }
    __syncthreads();
  }
  // The outputs of a chunk are stored when the next one's tiles have arrived: loads and stores
  // are waited for in one count, and stores issued between a chunk's loads and their use would
  // have to reach memory first.
  uint2 done[OT][VT];
  op += l16 * a.os[2] + g4;
  auto store_out = [&](int t) {
    const int n = min(kChunk, t1 - t);
#pragma unroll
    for (int x = 0; x < OT; ++x) {
      const int j = DW == 1 ? x : wd == 0 ? 3 * x : 1 + x;
#pragma unroll
      for (int v = 0; v < VT; ++v)
        if (16 * j + l16 < n && wv * CW + 16 * v + g4 < nc)
          *reinterpret_cast<uint2*>(op + (t + 16 * j) * a.os[2] + 16 * v) = done[x][v];
    }
  };
  int rq = at<DK>(l16, g4), rp = at<kChunk>(l16, g4);
  int ck = at<DK>(g4 + (l16 >> 2), drow + (l16 & 3) * 4), cv = at<DV>(g4 + (l16 >> 2), wv * CW + (l16 & 3) * 4);
  int buf = 0;
  for (int t = t0; t < t1; t += kChunk, buf ^= 1) {
    const int n = min(kChunk, t1 - t);
    // opaque, so that what is XORed from them is formed where it is used and not kept in registers
    // over the whole loop
    asm volatile("" : "+v"(rq), "+v"(rp), "+v"(ck), "+v"(cv));
    asm volatile("" : "+v"(gnext));         // arrived with the tiles, not after the next ones
    const bool mine = tv.nonfinite();       // (columns past d_v repeat others of the row)
    if (mine) dec[buf].bad = 1;
    if constexpr (kOut) {
      tq.trim(n, a.dk);
      tq.template store<true>(qt);
    }
    tk.trim(n, a.dk);
    tk.template store<true>(kt);
    tv.trim(n, nc);
    if constexpr (kHasV) tv.template store<false>(vt);
    if constexpr (kParts) {
      using TV = Tile<DV, NT>;
      const int row = tid / TV::kPer, c = tid % TV::kPer * 8;
#pragma unroll
      for (int i = 0; i < TV::kN; ++i) {
        uint4 part[PARTS];
        const float w = dec[buf].w[row + i * TV::kStep];
        if (mine) tv.template split<PARTS, true>(i, w, part);
        else tv.template split<PARTS, false>(i, w, part);
#pragma unroll
        for (int p = 0; p < PARTS; ++p)
          *reinterpret_cast<uint4*>(wt + p * kTileV + at<DV>(row + i * TV::kStep, c)) = part[p];
      }
    }
    if constexpr (kOut)
      if (t > t0) store_out(t - kChunk);
    __syncthreads();
    const Decays& D = dec[buf];
    // (the next tiles' loads are issued in three parts: all at once they would fill the memory
    // pipe and hold the waves up)
    const bool more = t + kChunk < t1;
    if (more) {
      fetch_v(t + kChunk);
      if (wave == NT / 64 - 1) {
        gsum += scan_decays(gnext, log2_scale, &dec[buf ^ 1]);
        gnext = log_decay(t + 2 * kChunk);
      }
      if (tid == 0) dec[buf ^ 1].bad = 0;
    }
    f32x4 O[4][VT];
    if constexpr (kOut) {
      // scores P^T = K Q^T, keys in the rows: a wave has one tile of 16 keys and meets the query
      // tiles from its own on (four waves), or half of them (eight), with it
      constexpr int JT = 16 / (NT / 64);    // query tiles a wave
      const int j0 = JT == 4 ? 0 : (wave >> 2) * 2;
      if (keys <= j0 + JT - 1) {
        const char* kk = kt + keys * kRows<DK>;
        const char* qq = qt + j0 * kRows<DK>;
        const int pj = (rp ^ (keys << 5)) + j0 * kRows<kChunk>;
        const f32x4 cs = *reinterpret_cast<const f32x4*>(&D.c[16 * keys + g4]);
        const f32x4 ls = *reinterpret_cast<const f32x4*>(&D.l[16 * keys + g4]);
        const int ahead = l16 - g4 + 16 * (j0 - keys);   // queries' lead over the lane's first key
        auto finish = [&](int j, const f32x4& p) {
          const float ct = D.c[16 * (j0 + j) + l16], lt = D.q[16 * (j0 + j) + l16];
          float x[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) x[r] = p[r] * __builtin_amdgcn_exp2f((ct - cs[r]) + (lt - ls[r]));
          if (j0 + j <= keys) {             // on the diagonal (or above it)
#pragma unroll
            for (int r = 0; r < 4; ++r) x[r] = ahead + 16 * j >= r ? x[r] : 0.f;
          }
          uint32_t u[2][2];
          split_pair<2, false>(x[0], x[1], &u[0][0], 2);
          split_pair<2, false>(x[2], x[3], &u[0][1], 2);
          const uint32_t m = low_mask(fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3]))));
          const int p0 = pj + j * kRows<kChunk>;
          *reinterpret_cast<uint2*>(pt + p0) = make_uint2(u[0][0], u[0][1]);
          *reinterpret_cast<uint2*>(pt + low_part(p0, j0 + j)) = make_uint2(u[1][0] & m, u[1][1] & m);
        };
        if constexpr (JT == 4) {
          bf16x8 kf[KS];
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) kf[ks] = row_operand(kk, rq, ks, 0);
#pragma unroll
          for (int j = 0; j < JT; ++j) {
            if (j0 + j < keys) continue;
            f32x4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) p = mfma(kf[ks], row_operand(qq, rq, ks, j * kRows<DK>), p);
            finish(j, p);
          }
        } else {                            // both tiles at once: no room for all of the keys' operands
          f32x4 p[JT];
#pragma unroll
          for (int j = 0; j < JT; ++j) p[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            const bf16x8 kf = row_operand(kk, rq, ks, 0);
#pragma unroll
            for (int j = 0; j < JT; ++j) p[j] = mfma(kf, row_operand(qq, rq, ks, j * kRows<DK>), p[j]);
          }
#pragma unroll
          for (int j = 0; j < JT; ++j) finish(j, p[j]);
        }
      }
      if (more) fetch_k(t + kChunk);
      // what the state in front of the chunk gives: O^T = S^T Q^T, scaled by 2^c of the query
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int v = 0; v < VT; ++v) O[j][v] = f32x4{0.f, 0.f, 0.f, 0.f};
      uint32_t mask[VT];
#pragma unroll
      for (int v = 0; v < VT; ++v) {
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < AT; ++i) top = fmaxf(fmaxf(fmaxf(top, fabsf(S[i][v][0])), fmaxf(fabsf(S[i][v][1]), fabsf(S[i][v][2]))), fabsf(S[i][v][3]));
        mask[v] = low_mask(top);
      }
#pragma unroll
      for (int ks = 0; ks < KS / DW; ++ks) {
        bf16x8 sf[2][VT];
#pragma unroll
        for (int v = 0; v < VT; ++v) {
          const f32x4 x = S[2 * ks][v], y = S[2 * ks + 1][v];
          uint32_t u[2][4];
          split_pair<2, false>(x[0], x[1], &u[0][0], 4);
          split_pair<2, false>(x[2], x[3], &u[0][1], 4);
          split_pair<2, false>(y[0], y[1], &u[0][2], 4);
          split_pair<2, false>(y[2], y[3], &u[0][3], 4);
          sf[0][v] = __builtin_bit_cast(bf16x8, make_uint4(u[0][0], u[0][1], u[0][2], u[0][3]));
          sf[1][v] = __builtin_bit_cast(bf16x8, make_uint4(u[1][0] & mask[v], u[1][1] & mask[v], u[1][2] & mask[v], u[1][3] & mask[v]));
        }
        // products that follow each other have different accumulators
        constexpr int JB = 4 / VT;
#pragma unroll
        for (int j0 = 0; j0 < 4; j0 += JB) {
          bf16x8 q[JB];
#pragma unroll
          for (int j = 0; j < JB; ++j) q[j] = row_operand(qt, rq ^ (drow * 2), ks, (j0 + j) * kRows<DK>);
#pragma unroll
          for (int p = 1; p >= 0; --p)
#pragma unroll
            for (int j = 0; j < JB; ++j)
#pragma unroll
              for (int v = 0; v < VT; ++v) O[j0 + j][v] = mfma(sf[p][v], q[j], O[j0 + j][v]);
        }
      }
      if constexpr (DW == 2) {              // tiles 0 and 3 are finished by wd 0, 1 and 2 by wd 1
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int v = 0; v < VT; ++v)
            swap[((wave * 2 + x) * VT + v) * 64 + lane] = wd == 0 ? O[1 + x][v] : O[3 * x][v];
      }
    }
    if (more) {
      if constexpr (kOut) fetch_q(t + kChunk);
      else fetch_k(t + kChunk);
    }
    // (the largest head has no register left for products started early)
    if constexpr (DK == 256) __builtin_amdgcn_sched_barrier(0);
    const bool bad = __builtin_amdgcn_readfirstlane(D.bad);   // (one for the block)
    bf16x8 vf[2][VT];
    if constexpr (kHasV)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int v = 0; v < VT; ++v) vf[ks][v] = col_operand<32 * DV>(vt, cv, ks, v);
    if (MODE != kLinOut || more) {
      // S <- a S + K^T (w V): the parts of w V in the same order of tokens as K^T
      const float dec64 = D.a;
#pragma unroll
      for (int i = 0; i < AT; ++i)
#pragma unroll
        for (int v = 0; v < VT; ++v) S[i][v] *= dec64;
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        if constexpr (DK == 256) __builtin_amdgcn_sched_barrier(0);
        bf16x8 wf[VT][PARTS];
        if constexpr (kParts) {
#pragma unroll
          for (int v = 0; v < VT; ++v)
#pragma unroll
            for (int p = 0; p < PARTS; ++p) wf[v][p] = col_operand<32 * DV>(wt + p * kTileV, cv, ks, v);
        } else {
          const f32x4 w0 = *reinterpret_cast<const f32x4*>(&D.w[32 * ks + g4]);
          const f32x4 w1 = *reinterpret_cast<const f32x4*>(&D.w[32 * ks + 16 + g4]);
          auto parts = [&](auto safe) {
#pragma unroll
            for (int v = 0; v < VT; ++v) {
              const uint4 u = __builtin_bit_cast(uint4, vf[ks][v]);
              const uint32_t uu[4] = {u.x, u.y, u.z, u.w};
              uint32_t o[PARTS][4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float x = j < 2 ? w0[2 * j] : w1[2 * j - 4], y = j < 2 ? w0[2 * j + 1] : w1[2 * j - 3];
                split_pair<PARTS, decltype(safe)::value>(__uint_as_float(uu[j] << 16) * x, __uint_as_float(uu[j] & 0xffff0000u) * y, &o[0][j], 4);
              }
#pragma unroll
              for (int p = 0; p < PARTS; ++p) wf[v][p] = __builtin_bit_cast(bf16x8, make_uint4(o[p][0], o[p][1], o[p][2], o[p][3]));
            }
          };
          if (bad) parts(std::true_type{});
          else parts(std::false_type{});
        }
        // four state tiles at a time, part by part: products that follow each other have
        // different accumulators
        constexpr int B = AT < 4 ? AT : 4;
#pragma unroll
        for (int i0 = 0; i0 < AT; i0 += B) {
          bf16x8 kf[B];
#pragma unroll
          for (int i = 0; i < B; ++i) kf[i] = col_operand<kRows<DK>>(kt, ck, ks, i0 + i);
#pragma unroll
          for (int p = PARTS - 1; p >= 0; --p)
#pragma unroll
            for (int i = 0; i < B; ++i)
#pragma unroll
              for (int v = 0; v < VT; ++v) S[i0 + i][v] = mfma(kf[i], wf[v][p], S[i0 + i][v]);
        }
      }
    }
    // The score tile and the shares are whole, and the tiles of Q, K and V are free: what follows
    // reads neither, and the next chunk's tiles may be written meanwhile.
    __syncthreads();
    if constexpr (kOut) {
#pragma unroll
      for (int x = 0; x < OT; ++x) {
        const int j = DW == 1 ? x : wd == 0 ? 3 * x : 1 + x;
        const float e = D.e[16 * j + l16];
        f32x4 o[VT];
#pragma unroll
        for (int v = 0; v < VT; ++v) {
          if constexpr (DW == 2) {
            o[v] = wd == 0 ? O[3 * x][v] : O[1 + x][v];
            o[v] += swap[(((wave ^ VW) * 2 + x) * VT + v) * 64 + lane];
          } else {
            o[v] = O[x][v];
          }
          o[v] *= e;
        }
        const int tt = 16 * j + l16;
        if (!bad) {
          // keys up to the query's tile: 32 or 64
#pragma unroll
          for (int ks = 0; ks < 2; ++ks)
            if (ks <= j / 2) {
              const bf16x8 lo = row_operand(pt, rp, j < 2 ? 1 : ks, (j < 2 ? j : j + 2) * kRows<kChunk>);
              const bf16x8 hi = row_operand(pt, rp, ks, j * kRows<kChunk>);
#pragma unroll
              for (int v = 0; v < VT; ++v) o[v] = mfma(vf[ks][v], lo, o[v]);
#pragma unroll
              for (int v = 0; v < VT; ++v) o[v] = mfma(vf[ks][v], hi, o[v]);
            }
        } else {
          // 0 times a NaN or an infinity of a later token must not reach this one: the same
          // sums, over the tokens up to the query's only
#pragma unroll 1
          for (int k = 0; k < 16 * j + 16; ++k) {
            const int at_p = at_gap<kChunk>(tt, k);
            const float p = bf16_to_f32(*reinterpret_cast<const uint16_t*>(pt + at_p)) +
                            bf16_to_f32(*reinterpret_cast<const uint16_t*>(pt + low_part(at_p, j)));
#pragma unroll
            for (int v = 0; v < VT; ++v) {
              const uint2 u = *reinterpret_cast<const uint2*>(vt + at<DV>(k, wv * CW + 16 * v + g4));
              const float y[4] = {__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                                  __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u)};
#pragma unroll
              for (int r = 0; r < 4; ++r) o[v][r] = k <= tt ? fmaf(p, y[r], o[v][r]) : o[v][r];
            }
          }
        }
#pragma unroll
        for (int v = 0; v < VT; ++v) {
          if (a.scale < 0.f) o[v] = -o[v];
          done[x][v] = make_uint2(pack_bf16x2(o[v][0], o[v][1]), pack_bf16x2(o[v][2], o[v][3]));
        }
      }
      if (bad) __syncthreads();             // (the V tile was read here)
    }
  }
  if constexpr (kOut)
    if (t0 < t1) store_out(t0 + (t1 - t0 - 1) / kChunk * kChunk);
  float* to = nullptr;
  if (MODE == kLinWhole && keep && one) to = a.state_out + (static_cast<int64_t>(slot) * a.H + h) * sh;
  if (MODE == kLinState) {
    const int64_t i = lin_segment(a, s, row0, seg) * a.H + h;
    to = a.seg_state + i * sh;
    if (c0 == 0 && wave == NT / 64 - 1 && lane == 0) a.seg_decay[i] = exp2f(static_cast<float>(gsum));
  }
  if (to) {
#pragma unroll
    for (int i = 0; i < AT; ++i)
#pragma unroll
      for (int j = 0; j < VT; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int d = drow + 16 * i + g4 + r, v = vcol + 16 * j;
          if (d < a.dk && v < a.dv) to[static_cast<int64_t>(d) * a.dv + v] = S[i][j][r];
        }
  }
}

// Columns a block. With d_k above 128, 128 where d_v has them: each chunk's Q and K are then read
// from memory and LDS for twice the columns (8192 tokens, 16 heads of 256 x 512: 350 us, against 605
// us with 64 columns; 8 sequences of 2048 tokens, in one pass: 651 and 637 us). Below, 64: more
// blocks a CU hide more of the waits between a chunk's phases (13 packed sequences of 32 heads of 64 x
// 128, with one part of each score and state: 140 us, against 168 us with 128 columns).
int columns(const LinArgs& a) { return a.dk > 128 && a.dv > 64 ? 128 : 64; }

template <int DK, int CW, int VW, int DW, LinMode MODE>
hipError_t launch_t(const LinArgs& a, hipStream_t st) {
  const int slices = (a.dv + VW * CW - 1) / (VW * CW);
  const bool rest = a.T > 0 && a.zero_rest && MODE != kLinState;
  const dim3 grid = lin_grid(a, a.H * slices, rest), block(64 * VW * DW);
  hipLaunchKernelGGL((lin_chunks<DK, CW, VW, DW, MODE>), grid, block, 0, st, a);
  return hipGetLastError();
}

template <LinMode MODE>
hipError_t launch_mode(const LinArgs& a, hipStream_t st) {
  if (a.dk <= 64) return launch_t<64, 16, 4, 1, MODE>(a, st);
  if (a.dk <= 128) return launch_t<128, 16, 4, 1, MODE>(a, st);
  if (columns(a) == 128) return launch_t<256, 32, 4, 2, MODE>(a, st);
  return launch_t<256, 16, 4, 2, MODE>(a, st);
}

}  // namespace

int lin_mfma_blocks(const LinArgs& a) {
  const int w = columns(a);
  return a.H * ((a.dv + w - 1) / w);
}

hipError_t launch_lin_mfma(const LinArgs& a, LinMode mode, hipStream_t st) {
  if (mode == kLinWhole) return launch_mode<kLinWhole>(a, st);
  if (mode == kLinState) return launch_mode<kLinState>(a, st);
  return launch_mode<kLinOut>(a, st);
}

}  // namespace rn
