// Short causal convolution of every channel with its own K weights, K <= 8:
//     u_t = b + sum_j w_j x_{t-K+1+j},     out = u, or u sigmoid(u),
// with the K - 1 inputs before a sequence's first token from its state (zeros without one), and its last
// K - 1 inputs left as the new state. Backward, with du = dout act'(u):
//     dx_t = sum_j w_j du_{t+K-1-j},   dw_j = sum_t du_t x_{t-K+1+j},   db = sum_t du_t.
//
// Bound by HBM: x is read once and out written once (14001 packed tokens of 4096 channels, bf16, K = 4 and
// u sigmoid(u): 56 us, 4.1 TB/s; gradients of 2 x 4095: a call 66 us, 5 of them the weights' sums, 3.3 TB/s in the
// rest; in float32 96 us, 4.4 TB/s). A thread
// takes 16 bytes of channels (8 of bf16 backward, whose sums take registers) and a run of tokens, whose rows it
// asks for at once; those before and behind it are its neighbours' and come from a cache.
#include <algorithm>

#include "norm_rows.h"
#include "rn_kernels.h"
#include "sequences.h"

namespace rn {
namespace {

// Tokens a thread takes, forward and backward, whose rows it asks for at once (14001 packed tokens of
// 4096 channels bf16, K = 4, with runs of 8 tokens 56 us, of 16 59, of 4 75; gradients of 2 x 4095 tokens with
// runs of 8 and three blocks a CU 65 us, of 16 in two 72; now 66, sums leaving out tokens behind the last).
constexpr int kRun = 8, kBackRun = 8;

struct ConvArgs {
  Seqs q;
  int32_t D, K, n_slots;
  int32_t lanes;                          // lanes along channels: a power of two, 256 / lanes runs a block
  bool silu, zero_rest;
  int64_t xs[2], os[2], ds[2];            // sequence and token strides: x, out / dout, dx
  const int32_t* slots;
  const void* x;
  const float* w;                         // [D][K]
  const float* b;                         // [D] or null
  const void* state_in;                   // [slots or S][K - 1][D] or null
  void* state_out;
  void* out;
  const void* dout;
  void* dx;
  const float* dstate_out;                // [S][K - 1][D] or null
  float* dstate_in;
  float* part;                            // [grid rows][K + 1][D]: sums of dw and db, or null
};

template <int K, int V, Fit FIT>
__device__ __forceinline__ void conv_weights(const ConvArgs& a, int c, float (*w)[K], float* b) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const bool there = FIT != kOdd || c + v < a.D;
#pragma unroll
    for (int j = 0; j < K; ++j) w[v][j] = there ? a.w[static_cast<int64_t>(c + v) * K + j] : 0.f;
    b[v] = there && a.b ? a.b[c + v] : 0.f;
  }
}

template <int DT, int K, int V, Fit FIT>
__global__ void __launch_bounds__(256) conv_rows(ConvArgs a) {
  Span p;
  if (!seq_place(a.q, blockIdx.y + static_cast<int64_t>(blockIdx.z) * gridDim.y, &p)) return;
  const int c = (blockIdx.x * a.lanes + threadIdx.x % a.lanes) * V, left = a.D - c;
  if (c >= a.D) return;
  const int run = threadIdx.x / a.lanes;
  const int64_t t0 = static_cast<int64_t>(p.piece) * a.q.len + run * kRun;
  const bool head = p.piece == 0 && run == 0;
  if (t0 >= p.own && !head) return;
  const int64_t xb = seq_base(a.q, p, a.xs[0], a.xs[1]) + c, ob = seq_base(a.q, p, a.os[0], a.os[1]) + c;
  // x[i]: token t0 - (K - 1) + i
  Raw<DT, V, FIT> x[kRun + K - 1];
#pragma unroll
  for (int i = 0; i < kRun + K - 1; ++i) {
    const int64_t t = t0 - (K - 1) + i;
    if (t >= 0 && t < p.len) x[i].load(a.x, xb + t * a.xs[1], left);
    else x[i].clear();
  }
  if (head && p.s < a.q.S) {
    const int slot = seq_slot(a.slots, a.n_slots, p.s);
    const int64_t sb = static_cast<int64_t>(slot) * (K - 1) * a.D + c;
    if (slot >= 0 && a.state_in) {
#pragma unroll
      for (int i = 0; i < K - 1; ++i) x[i].load(a.state_in, sb + static_cast<int64_t>(i) * a.D, left);
    }
    // the same thread has read the state that it now replaces (the two may be one buffer)
    if (slot >= 0 && a.state_out) {
#pragma unroll
      for (int i = 0; i < K - 1; ++i) {
        const int64_t t = static_cast<int64_t>(p.len) - (K - 1) + i;
        Raw<DT, V, FIT> y;
        y.clear();
        if (t >= 0) {
          y.load(a.x, xb + t * a.xs[1], left);
        } else {
#pragma unroll
          for (int k = 0; k < K - 1; ++k)
            if (k == t + K - 1) y = x[k];
        }
        y.store(a.state_out, sb + static_cast<int64_t>(i) * a.D, left);
      }
    }
  }
  float w[V][K], b[V];
  conv_weights<K, V, FIT>(a, c, w, b);
#pragma unroll
  for (int i = 0; i < kRun; ++i) {
    const int64_t t = t0 + i;
    float u[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      u[v] = b[v];
#pragma unroll
      for (int j = 0; j < K; ++j) u[v] = fmaf(w[v][j], x[i + j].value(v), u[v]);
      if (a.silu) u[v] = swishf(u[v]);
    }
    if (t < p.len) store<DT, V, FIT>(a.out, ob + t * a.os[1], left, u);
    else if (a.zero_rest && t < p.own) {
      Raw<DT, V, FIT> z;
      z.clear();
      z.store(a.out, ob + t * a.os[1], left);
    }
  }
}

// One token a sequence; a thread's channels' state is read and moved up by one row.
template <int DT, int K, int V, Fit FIT>
__global__ void __launch_bounds__(256) conv_step(ConvArgs a) {
  const int s = blockIdx.y * (256 / a.lanes) + threadIdx.x / a.lanes;
  const int c = (blockIdx.x * a.lanes + threadIdx.x % a.lanes) * V, left = a.D - c;
  if (s >= a.q.S || c >= a.D) return;
  const int slot = seq_slot(a.slots, a.n_slots, s);
  const int64_t ob = s * a.os[0] + c, sb = static_cast<int64_t>(slot) * (K - 1) * a.D + c;
  float u[V];
  if (slot < 0) {
#pragma unroll
    for (int v = 0; v < V; ++v) u[v] = 0.f;
    store<DT, V, FIT>(a.out, ob, left, u);
    return;
  }
  Raw<DT, V, FIT> x[K];
#pragma unroll
  for (int i = 0; i < K - 1; ++i) x[i].load(a.state_in, sb + static_cast<int64_t>(i) * a.D, left);
  x[K - 1].load(a.x, s * a.xs[0] + c, left);
  float w[V][K], b[V];
  conv_weights<K, V, FIT>(a, c, w, b);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    u[v] = b[v];
#pragma unroll
    for (int j = 0; j < K; ++j) u[v] = fmaf(w[v][j], x[j].value(v), u[v]);
    if (a.silu) u[v] = swishf(u[v]);
  }
  store<DT, V, FIT>(a.out, ob, left, u);
#pragma unroll
  for (int i = 0; i < K - 1; ++i) x[i + 1].store(a.state_out, sb + static_cast<int64_t>(i) * a.D, left);
}

// A thread takes its runs of tokens in turn (pieces gridDim.y apart) and sums dw and db over them; the
// runs of a block are added in their order, the blocks' sums by conv_reduce.
template <int DT, int K, int V, Fit FIT>
__global__ void __launch_bounds__(256, DT == RN_BF16 && K <= 5 ? 3 : 2) conv_backward(ConvArgs a) {
  __shared__ float merge[256 * V];
  const int c = (blockIdx.x * a.lanes + threadIdx.x % a.lanes) * V, left = a.D - c;
  const int run = threadIdx.x / a.lanes;
  const bool mine = c < a.D;
  float w[V][K], b[V], dw[K][V], db[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    b[v] = db[v] = 0.f;
#pragma unroll
    for (int j = 0; j < K; ++j) w[v][j] = dw[j][v] = 0.f;
  }
  if (mine) conv_weights<K, V, FIT>(a, c, w, b);
  const int64_t pieces = seq_pieces(a.q);
  for (int64_t piece = blockIdx.y; piece < pieces; piece += gridDim.y) {
    Span p;
    if (!seq_place(a.q, piece, &p) || !mine) continue;
    const int64_t t0 = static_cast<int64_t>(p.piece) * a.q.len + run * kBackRun;
    const bool head = p.piece == 0 && run == 0;
    if (t0 >= p.own && !head) continue;
    const int64_t xb = seq_base(a.q, p, a.xs[0], a.xs[1]) + c, ob = seq_base(a.q, p, a.os[0], a.os[1]) + c,
                  db0 = seq_base(a.q, p, a.ds[0], a.ds[1]) + c;
    const bool real = p.s < a.q.S;
    const int64_t sb = static_cast<int64_t>(p.s) * (K - 1) * a.D + c;     // of a state's row 0
    // x[i]: token t0 - (K - 1) + i; g[i]: dout of token t0 + i. All at once, from rows inside the sequence, and
    // zeros where the token is not.
    Raw<DT, V, FIT> x[kBackRun + 2 * K - 2], g[kBackRun + K - 1];
#pragma unroll
    for (int i = 0; i < kBackRun + 2 * K - 2; ++i) x[i].clear();
#pragma unroll
    for (int i = 0; i < kBackRun + K - 1; ++i) g[i].clear();
    if (p.len > 0) {
      auto row = [&](int64_t t) { return min(max(t, int64_t(0)), static_cast<int64_t>(p.len) - 1); };
#pragma unroll
      for (int i = 0; i < kBackRun + 2 * K - 2; ++i) x[i].load(a.x, xb + row(t0 - (K - 1) + i) * a.xs[1], left);
#pragma unroll
      for (int i = 0; i < kBackRun + K - 1; ++i) g[i].load(a.dout, ob + row(t0 + i) * a.os[1], left);
      if (t0 < K - 1 || t0 + kBackRun + K - 1 > p.len) {
#pragma unroll
        for (int i = 0; i < kBackRun + 2 * K - 2; ++i)
          if (t0 - (K - 1) + i < 0 || t0 - (K - 1) + i >= p.len) x[i].clear();
      }
    }
    if (head && real && a.state_in) {
#pragma unroll
      for (int i = 0; i < K - 1; ++i) x[i].load(a.state_in, sb + static_cast<int64_t>(i) * a.D, left);
    }
    float du[kBackRun + K - 1][V];
#pragma unroll
    for (int i = 0; i < kBackRun + K - 1; ++i) {
      const int64_t t = t0 + i, at = t - (K - 1);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float d = g[i].value(v);
        if (a.silu) {
          float u = b[v];
#pragma unroll
          for (int j = 0; j < K; ++j) u = fmaf(w[v][j], x[i + j].value(v), u);
          const float sg = __builtin_amdgcn_rcpf(1.0f + __expf(-u));
          d *= sg * fmaf(u, 1.0f - sg, 1.0f);
        }
        du[i][v] = d = t < p.len ? d : 0.f;
      }
      if (i < kBackRun && t < p.len) {       // (no 0 x of a token behind the last one: x may be infinite)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          db[v] += du[i][v];
#pragma unroll
          for (int j = 0; j < K; ++j) dw[j][v] = fmaf(du[i][v], x[i + j].value(v), dw[j][v]);
        }
      }
      // dx of token t - (K - 1), a row of the state where it is before the first
      if (i >= K - 1 || head) {
        float dx[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          dx[v] = 0.f;
#pragma unroll
          for (int j = 0; j < K; ++j)
            if (i - j >= 0) dx[v] = fmaf(w[v][j], du[i - j < 0 ? 0 : i - j][v], dx[v]);
        }
        // the final state's gradient reaches the tokens that it holds
        const int64_t k = at - (static_cast<int64_t>(p.len) - (K - 1));
        if (real && a.dstate_out && k >= 0 && k < K - 1) {
          float more[V];
          load<RN_F32, V, FIT>(a.dstate_out, sb + k * a.D, left, more);
#pragma unroll
          for (int v = 0; v < V; ++v) dx[v] += more[v];
        }
        if (at < 0) {
          if (real && a.dstate_in) store<RN_F32, V, FIT>(a.dstate_in, sb + (at + K - 1) * a.D, left, dx);
        } else if (at < p.len) {
          store<DT, V, FIT>(a.dx, db0 + at * a.ds[1], left, dx);
        } else if (at < p.own && a.zero_rest) {
          Raw<DT, V, FIT> z;
          z.clear();
          z.store(a.dx, db0 + at * a.ds[1], left);
        }
      }
    }
  }
  if (!a.part) return;
  const int runs = 256 / a.lanes;
  float* part = a.part + static_cast<int64_t>(blockIdx.y) * (K + 1) * a.D;
#pragma unroll
  for (int j = 0; j <= K; ++j) {
#pragma unroll
    for (int v = 0; v < V; ++v) merge[v * 256 + threadIdx.x] = j < K ? dw[j < K ? j : 0][v] : db[v];
    __syncthreads();
    for (int i = threadIdx.x; i < a.lanes * V; i += 256) {
      const int v = i / a.lanes, l = i % a.lanes, col = (blockIdx.x * a.lanes + l) * V + v;
      float s = 0.f;
      for (int r = 0; r < runs; ++r) s += merge[v * 256 + r * a.lanes + l];
      if (col < a.D) part[static_cast<int64_t>(j) * a.D + col] = s;
    }
    __syncthreads();
  }
}

// dweight [D][K] and dbias [D] from the blocks' sums [rows][K + 1][D], in a fixed order.
__global__ void __launch_bounds__(1024) conv_reduce(const float* part, int rows, int D, int K, float* dw, float* db) {
  __shared__ float red[32][33];
  const int64_t cols = static_cast<int64_t>(K + 1) * D;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + (threadIdx.x & 31);
  const int grp = threadIdx.x >> 5;
  float s = 0.f;
  if (col < cols) {
#pragma unroll 8
    for (int i = grp; i < rows; i += 32) s += part[i * cols + col];
  }
  red[grp][threadIdx.x & 31] = s;
  __syncthreads();
  if (grp == 0 && col < cols) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += red[i][threadIdx.x];
    const int64_t j = col / D, d = col - j * D;
    if (j < K) { if (dw) dw[d * K + j] = s; }
    else if (db) db[d] = s;
  }
}

// Channels a thread: 16 bytes of x forward, half as many of bf16 backward (whose sums take registers).
template <int DT> constexpr int width(bool back) { return DT == RN_BF16 && !back ? 8 : 4; }
int lanes_of(int D, int V) {
  int n = 1;
  while (n < 64 && n * V < D) n *= 2;
  return n;
}
int tokens_a_block(const ConvCall& c) {
  const int V = c.dt == RN_BF16 && !c.backward ? 8 : 4;
  return 256 / lanes_of(c.D, V) * (c.backward ? kBackRun : kRun);
}
Seqs seqs_of(const ConvCall& c) {
  Seqs q{c.S, c.N, c.T, 0, 0, c.cu, c.lens};
  seq_cut(&q, tokens_a_block(c));
  return q;
}
// Rows of blocks along the tokens in the backward: each leaves (K + 1) D sums.
int64_t backward_rows(const ConvCall& c) { return std::min<int64_t>(seq_pieces(seqs_of(c)), 128); }

template <int DT, int K, Fit FIT>
hipError_t launch_fit(const ConvCall& c, ConvArgs a, hipStream_t st) {
  if (c.backward) {
    constexpr int V = width<DT>(true);
    a.lanes = lanes_of(c.D, V);
    const int64_t x = (c.D + static_cast<int64_t>(a.lanes) * V - 1) / (static_cast<int64_t>(a.lanes) * V);
    const int64_t rows = backward_rows(c);
    hipLaunchKernelGGL((conv_backward<DT, K, V, FIT>), dim3(static_cast<unsigned>(x), static_cast<unsigned>(rows)), dim3(256), 0, st, a);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && a.part) {
      hipLaunchKernelGGL(conv_reduce, dim3(static_cast<unsigned>((static_cast<int64_t>(K + 1) * c.D + 31) / 32)), dim3(1024), 0, st,
                         a.part, static_cast<int>(rows), c.D, K, c.dw, c.db);
      e = hipGetLastError();
    }
    return e;
  }
  constexpr int V = width<DT>(false);
  a.lanes = lanes_of(c.D, V);
  const int64_t x = (c.D + static_cast<int64_t>(a.lanes) * V - 1) / (static_cast<int64_t>(a.lanes) * V);
  if (c.step) {
    const int per = 256 / a.lanes;
    hipLaunchKernelGGL((conv_step<DT, K, V, FIT>), dim3(static_cast<unsigned>(x), (c.S + per - 1) / per), dim3(256), 0, st, a);
  } else {
    hipLaunchKernelGGL((conv_rows<DT, K, V, FIT>), seq_grid(a.q, x), dim3(256), 0, st, a);
  }
  return hipGetLastError();
}
template <int DT, int K>
hipError_t launch_k(const ConvCall& c, const ConvArgs& a, hipStream_t st) {
  return c.vec ? launch_fit<DT, K, kSome>(c, a, st) : launch_fit<DT, K, kOdd>(c, a, st);
}
template <int DT>
hipError_t launch_t(const ConvCall& c, const ConvArgs& a, hipStream_t st) {
  switch (c.K) {
    case 1: return launch_k<DT, 1>(c, a, st);
    case 2: return launch_k<DT, 2>(c, a, st);
    case 3: return launch_k<DT, 3>(c, a, st);
    case 4: return launch_k<DT, 4>(c, a, st);
    case 5: return launch_k<DT, 5>(c, a, st);
    case 6: return launch_k<DT, 6>(c, a, st);
    case 7: return launch_k<DT, 7>(c, a, st);
    default: return launch_k<DT, 8>(c, a, st);
  }
}

}  // namespace

size_t conv_backward_ws_bytes(const ConvCall& c) {
  return static_cast<size_t>(backward_rows(c)) * (c.K + 1) * c.D * sizeof(float);
}

hipError_t launch_short_conv(const ConvCall& c, hipStream_t st) {
  ConvArgs a;
  a.q = seqs_of(c);
  a.D = c.D; a.K = c.K; a.n_slots = c.n_slots; a.lanes = 0; a.silu = c.silu; a.zero_rest = c.zero_rest;
  for (int i = 0; i < 2; ++i) { a.xs[i] = c.xs[i]; a.os[i] = c.os[i]; a.ds[i] = c.ds ? c.ds[i] : 0; }
  a.slots = c.slots; a.x = c.x; a.w = c.w; a.b = c.b; a.state_in = c.state_in; a.state_out = c.state_out; a.out = c.out;
  a.dout = c.dout; a.dx = c.dx; a.dstate_out = c.dstate_out; a.dstate_in = c.dstate_in;
  a.part = c.dw || c.db ? static_cast<float*>(c.ws) : nullptr;
  return c.dt == RN_F32 ? launch_t<RN_F32>(c, a, st) : launch_t<RN_BF16>(c, a, st);
}

}  // namespace rn
