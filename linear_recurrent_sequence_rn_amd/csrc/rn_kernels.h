// Host-side launchers of the retention kernels (internal to the library).
#pragma once
#include <hip/hip_runtime.h>

#include "rn_device.h"

namespace rn {

hipError_t launch_generic_parallel(const CallArgs& a, int in_dt, int out_dt, const void* q,
                                   const void* k, const void* v, const void* gate, void* out,
                                   hipStream_t st);
hipError_t launch_generic_chunkwise(const CallArgs& a, int in_dt, int out_dt, const void* q,
                                    const void* k, const void* v, const void* gate,
                                    const float* s_in, float* s_out, void* out, float* ws,
                                    hipStream_t st);
hipError_t launch_decode_step(const CallArgs& a, int in_dt, int out_dt, const void* q,
                              const void* k, const void* v, const void* gate, float* state,
                              void* out, hipStream_t st);
hipError_t launch_groupnorm_gate(int B, int H, int N, int dv, int in_dt, int out_dt,
                                 const void* x, const void* gate, const float* w, const float* b,
                                 float eps, void* out, hipStream_t st);

// Fused MFMA chunkwise kernel (bf16 inputs, d_k = 256, d_v in {64,128,256,512}).
// Its workspace starts with the call's status word: these bits.
constexpr uint32_t kChunkwiseStatusTimeout = 1u;     // a cross-workgroup wait timed out
constexpr uint32_t kChunkwiseStatusNonFinite = 2u;   // a non-finite output or final state
bool chunkwise_mfma_supported(const CallArgs& a, int in_dt);
size_t chunkwise_mfma_ws_bytes(const CallArgs& a);
hipError_t launch_chunkwise_mfma(const CallArgs& a, int out_dt, const void* q, const void* k,
                                 const void* v, const void* gate, const float* s_in,
                                 float* s_out, void* out, void* ws, size_t ws_bytes,
                                 hipStream_t st);

// Chunk-parallel chunkwise pair: state snapshots, then outputs (bf16, d_k 256, d_v 512).
bool chunkwise_cp_supported(const CallArgs& a, int in_dt);
size_t chunkwise_cp_ws_bytes(const CallArgs& a);
hipError_t launch_chunkwise_cp(const CallArgs& a, int out_dt, const void* q, const void* k,
                               const void* v, const void* gate, const float* s_in, float* s_out,
                               void* out, void* ws, size_t ws_bytes, hipStream_t st);

// Segmented chunkwise schedule: segment-local states, a scan over segments, then the
// outputs of all chunks (bf16, d_k 256, d_v 512, one decay per head).
bool chunkwise_seg_supported(const CallArgs& a, int in_dt);
size_t chunkwise_seg_ws_bytes(const CallArgs& a);
hipError_t launch_chunkwise_seg(const CallArgs& a, int out_dt, const void* q, const void* k,
                                const void* v, const void* gate, const float* s_in, float* s_out,
                                void* out, void* ws, size_t ws_bytes, hipStream_t st);

// Gradients of the chunkwise form: f16-operand MFMA products with float32 accumulation for
// bf16 inputs whose d_k and d_v are multiples of 8, float32 products otherwise.
struct BwArgs {
  const void* q; const void* k; const void* v; const void* gate;
  const void* dout; const float* state_in; const float* dstate_out;
  void* dq; void* dk; void* dv; void* dgate; float* dstate_in;
  float* dgn_w; float* dgn_b;
};
size_t backward_ws_bytes(const CallArgs& a);
hipError_t launch_backward(const CallArgs& a, int in_dt, int out_dt, const BwArgs& x, void* ws,
                           hipStream_t st);
// Matrix-core path of the gradients (bf16 inputs, d_k and d_v multiples of 8; v, dv, dout,
// gate and dgate 16-byte and q, k 4-byte aligned).
bool backward_mfma_supported(const CallArgs& a, int in_dt);
size_t backward_mfma_ws_bytes(const CallArgs& a);
hipError_t launch_backward_mfma(const CallArgs& a, int out_dt, const BwArgs& x, void* ws,
                                hipStream_t st);

// MFMA parallel form (bf16 inputs, d_k = 256, d_v = 512).
bool parallel_mfma_supported(const CallArgs& a, int in_dt);
size_t parallel_mfma_ws_bytes(const CallArgs& a);
hipError_t launch_parallel_mfma(const CallArgs& a, int out_dt, const void* q, const void* k,
                                const void* v, const void* gate, void* out, void* ws,
                                hipStream_t st);

// Gated multi-scale retention layer: rocBLAS projections and output projection (return
// values are rocblas_status codes; 0 = success).
struct LayerArgs {
  int B, H, N, d_model, dk, dv;
};
int layer_project(const LayerArgs& L, const void* x, const void* w, int d, void* y,
                  hipStream_t stream);
int layer_output(const LayerArgs& L, const void* o, void* ot, const void* w_o, void* out,
                 int out_dtype, hipStream_t stream);
const char* blas_status_string(int status);

// ---- operators around retention (layernorm.hip, rotary.hip, linear_attention.hip) ----------
struct NormCall {
  int64_t rows;
  int32_t d;
  int in_dt, out_dt;
  float eps;
  bool backward;
  bool vec;                       // every row and pointer allows 16-byte accesses
  int64_t xs, rs, ss, os;         // row strides: x, residual / dsum, sum_out / dx, out / dout
  const void* x;
  const void* r;
  const float* w;
  const float* b;
  void* sum;
  void* out;
  const void* dout;
  float* dw;
  float* db;
  void* ws;
};
size_t norm_backward_ws_bytes(const NormCall& n);
hipError_t launch_layernorm(const NormCall& n, hipStream_t st);

struct RmsCall {
  int64_t rows;
  int32_t d, group;
  int in_dt, out_dt;
  float eps;
  bool backward;
  bool vec;                       // every row and pointer allows whole pieces
  int64_t xs, rs, ss, os, cs;     // row strides: x, residual / dsum, sum_out / dx, out / dout, scale
  const void* x;
  const void* r;
  const float* w;
  void* sum;
  void* out;
  float* scale;
  const void* dout;
  float* dw;
  void* ws;
};
size_t rms_backward_ws_bytes(const RmsCall& n);
hipError_t launch_rmsnorm(const RmsCall& n, hipStream_t st);

constexpr int kMaxRot = 256;
struct RotaryCall {
  int32_t B, N, Hq, Hk, d, rot;
  int dt;
  bool half, inverse, pos_token;
  float magnitude;
  int64_t pos0;
  const int64_t* pos;
  const double* theta;            // host
  const int64_t *qs, *ks, *qos, *kos;   // host [3]: batch, head, token
  const void* q;
  const void* k;
  void* q_out;
  void* k_out;
};
hipError_t launch_rotary(const RotaryCall& c, hipStream_t st);

struct LinCall {
  int32_t S, N, H, Hq, Hk, Hv, dk, dv;
  int in_dt, out_dt;
  bool generic, zero_rest;
  float scale;
  int64_t T;
  int32_t n_slots;
  const int64_t *qs, *ks, *vs, *gs, *os;   // host [3]: sequence, head, token
  const int32_t* cu;
  const int32_t* lens;
  const int32_t* slots;
  const void* q;
  const void* k;
  const void* v;
  const float* g;
  const float* state_in;
  float* state_out;
  void* out;
  void* ws;
};
size_t lin_ws_bytes(const LinCall& c);
hipError_t launch_linear_step(const LinCall& c, hipStream_t st);
hipError_t launch_linear_chunked(const LinCall& c, hipStream_t st);

struct ConvCall {
  int32_t S, N, D, K, n_slots;
  int64_t T;
  int dt;
  bool silu, zero_rest, backward, step;
  bool vec;                       // every row and pointer allows 16-byte accesses
  const int64_t *xs, *os, *ds;    // host [2]: sequence and token strides of x, out / dout, dx
  const int32_t* cu;
  const int32_t* lens;
  const int32_t* slots;
  const void* x;
  const float* w;
  const float* b;
  const void* state_in;
  void* state_out;
  void* out;
  const void* dout;
  void* dx;
  const float* dstate_out;
  float* dstate_in;
  float* dw;
  float* db;
  void* ws;
};
size_t conv_backward_ws_bytes(const ConvCall& c);
hipError_t launch_short_conv(const ConvCall& c, hipStream_t st);

struct ScanCall {
  int32_t S, N, D, n, G, n_slots;
  int64_t T;
  int type;
  bool softplus, zero_rest;
  const int64_t *xs, *dts, *zs, *os;   // host [2]: sequence and token strides
  const int64_t *bs, *cs;              // host [3]: sequence, group and token strides
  const int32_t* cu;
  const int32_t* lens;
  const int32_t* slots;
  const void* x;
  const void* dt;
  const void* z;
  const void* b;
  const void* c;
  const float* A;
  const float* skip;
  const float* bias;
  const float* state_in;
  float* state_out;
  void* out;
  void* ws;
};
size_t scan_ws_bytes(const ScanCall& c);
hipError_t launch_selective_scan(const ScanCall& c, hipStream_t st);
hipError_t launch_selective_step(const ScanCall& c, hipStream_t st);

struct ScanGrads {                // the call's out strides are those of dout
  const int64_t *dxs, *ddts, *dzs, *dbs, *dcs;   // host, as the inputs'
  const void* dout;
  const float* dstate_out;
  void* dx;
  void* ddt;
  void* dz;
  void* db;
  void* dc;
  float* dA;
  float* dskip;
  float* dbias;
  float* dstate_in;
};
size_t scan_backward_ws_bytes(const ScanCall& c);
hipError_t launch_selective_backward(const ScanCall& c, const ScanGrads& g, hipStream_t st);

// Records the message of a failed call (rn_last_error) and returns its status.
rn_status fail(rn_status s, const char* fmt, ...);
rn_status hip_status(hipError_t e, const char* what);
void clear_error();

}  // namespace rn
