// lynx_api_adapter.cu -- the C ABI's entry points for the weight in 4 bits, the
// 8-bit activation checkpoint, the backward pass, layer norm and the activation's
// gradient: argument checks and launches.  As everywhere, a failed check launches
// nothing.
#include <cmath>
#include <cstring>
#include <initializer_list>

#include "lynx.h"
#include "lynx_internal.h"

using namespace lynx;

namespace {

constexpr int64_t kMaxExtent = int64_t(1) << 30;

bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

template <typename... P>
bool any_misaligned(P... p) {
  return (misaligned(p) || ...);
}

template <typename... P>
bool any_null(P... p) {
  return ((p == nullptr) || ...);
}

bool rows_ok(int64_t M) { return M >= 1 && M <= kMaxExtent; }
bool k_ok(int64_t K) { return K >= 64 && K % 64 == 0 && K <= kMaxExtent; }
bool n_ok(int64_t N) { return N >= 8 && N % 8 == 0 && N <= kMaxExtent; }
bool group_ok(int64_t K, int group) { return (group == 32 || group == 64 || group == 128) && K % group == 0; }
bool rank_ok(int64_t r) { return lynx_lora_rank_supported(r) != 0; }
bool norm_cols_ok(int64_t K) { return K >= 8 && K % 8 == 0 && K <= kLayerNormMaxCols; }
bool eps_ok(float eps) { return eps >= 0.f && std::isfinite(eps); }
bool format_ok(int format) { return format == LYNX_CKPT8_INT8 || format == LYNX_CKPT8_E4M3; }

int status_of(cudaError_t e) { return e == cudaSuccess ? LYNX_OK : LYNX_ERR_CUDA; }

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// A and B (or dT and A) both or neither; r then a supported rank, else 0 or one
int check_branch(const void* a, const void* b, int64_t r) {
  if ((a == nullptr) != (b == nullptr)) return LYNX_ERR_INVALID_ARG;
  if ((a != nullptr || r != 0) && !rank_ok(r)) return LYNX_ERR_UNSUPPORTED_SHAPE;
  return LYNX_OK;
}

struct Span {
  const void* p;  // null: not there
  uint64_t bytes;
};

bool overlap(const Span& a, const Span& b) {
  const auto x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x != 0 && y != 0 && x < y + b.bytes && y < x + a.bytes;
}

// What a call writes must overlap neither what it reads nor its other outputs: its
// kernels read and write in an order that only the shape fixes.
bool any_overlap(std::initializer_list<Span> out, std::initializer_list<Span> in) {
  for (const Span* o = out.begin(); o != out.end(); ++o) {
    for (const Span& i : in)
      if (overlap(*o, i)) return true;
    for (const Span* q = out.begin(); q != o; ++q)
      if (overlap(*o, *q)) return true;
  }
  return false;
}

uint64_t bytes_of(int64_t rows, int64_t cols, int size) {
  return static_cast<uint64_t>(rows) * static_cast<uint64_t>(cols) * static_cast<uint64_t>(size);
}

}  // namespace

extern "C" {

size_t lynx_w4_bytes(int64_t N, int64_t K) {
  if (N <= 0 || K <= 0) return 0;
  return static_cast<size_t>(N) * static_cast<size_t>(K) / 2;
}

int lynx_w4_quantize(const void* W, int64_t N, int64_t K, int group, void* Wq, void* scales, void* zeros,
                     void* stream) {
  if (any_null(W, Wq, scales)) return LYNX_ERR_INVALID_ARG;
  if (!n_ok(N) || !k_ok(K) || !group_ok(K, group)) return LYNX_ERR_UNSUPPORTED_SHAPE;
  if (any_misaligned(W, Wq, scales, zeros)) return LYNX_ERR_MISALIGNED;
  if (any_overlap({{Wq, bytes_of(N, K / 2, 1)}, {scales, bytes_of(K / group, N, 2)}, {zeros, bytes_of(K / group, N, 1)}},
                  {{W, bytes_of(N, K, 2)}}))
    return LYNX_ERR_INVALID_ARG;
  return status_of(launch_w4_quantize(W, N, K, group, Wq, scales, zeros, static_cast<cudaStream_t>(stream)));
}

int lynx_w4_dequantize(const void* Wq, const void* scales, const void* zeros, int64_t N, int64_t K, int group,
                       void* W, void* stream) {
  if (any_null(Wq, scales, W)) return LYNX_ERR_INVALID_ARG;
  if (!n_ok(N) || !k_ok(K) || !group_ok(K, group)) return LYNX_ERR_UNSUPPORTED_SHAPE;
  if (any_misaligned(W, Wq, scales, zeros)) return LYNX_ERR_MISALIGNED;
  if (any_overlap({{W, bytes_of(N, K, 2)}}, {{Wq, bytes_of(N, K / 2, 1)},
                                             {scales, bytes_of(K / group, N, 2)},
                                             {zeros, bytes_of(K / group, N, 1)}}))
    return LYNX_ERR_INVALID_ARG;
  return status_of(launch_w4_dequantize(Wq, scales, zeros, N, K, group, W, static_cast<cudaStream_t>(stream)));
}

int64_t lynx_linear_w4_max_rows(void) { return LYNX_LINEAR_W4_MAX_ROWS; }

size_t lynx_linear_w4_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t r) {
  (void)N;
  if (M <= 0 || K <= 0 || r <= 0) return 0;
  return align256(static_cast<size_t>(M) * static_cast<size_t>(r) * 4);
}

int lynx_linear_w4(const void* X, const void* Wq, const void* scales, const void* zeros, const void* bias,
                   const void* A, const void* B, int64_t M, int64_t N, int64_t K, int64_t r, int group, int act,
                   void* Y, void* workspace, size_t workspace_bytes, void* stream) {
  return lynx_linear_w4_residual(X, Wq, scales, zeros, bias, A, B, nullptr, M, N, K, r, group, act, Y, workspace,
                                 workspace_bytes, stream);
}

int lynx_linear_w4_residual(const void* X, const void* Wq, const void* scales, const void* zeros, const void* bias,
                            const void* A, const void* B, const void* R, int64_t M, int64_t N, int64_t K, int64_t r,
                            int group, int act, void* Y, void* workspace, size_t workspace_bytes, void* stream) {
  static_assert(kLinearW4MaxRows == LYNX_LINEAR_W4_MAX_ROWS, "");
  if (any_null(X, Wq, scales, Y)) return LYNX_ERR_INVALID_ARG;
  if (act != LYNX_ACT_NONE && act != LYNX_ACT_GELU_TANH) return LYNX_ERR_INVALID_ARG;
  if (const int st = check_branch(A, B, r)) return st;
  if (M < 1 || M > LYNX_LINEAR_W4_MAX_ROWS || !n_ok(N) || !k_ok(K) || !group_ok(K, group))
    return LYNX_ERR_UNSUPPORTED_SHAPE;
  if (any_misaligned(X, Wq, scales, zeros, bias, A, B, R, Y, workspace)) return LYNX_ERR_MISALIGNED;
  if (A != nullptr) {
    if (workspace == nullptr) return LYNX_ERR_INVALID_ARG;
    if (workspace_bytes < lynx_linear_w4_workspace_bytes(M, N, K, r)) return LYNX_ERR_WORKSPACE_TOO_SMALL;
  }
  const Span ws = {A != nullptr ? workspace : nullptr, lynx_linear_w4_workspace_bytes(M, N, K, r)};
  if (any_overlap({{Y, bytes_of(M, N, 2)}, ws},
                  {{X, bytes_of(M, K, 2)},
                   {Wq, bytes_of(N, K / 2, 1)},
                   {scales, bytes_of(K / group, N, 2)},
                   {zeros, bytes_of(K / group, N, 1)},
                   {bias, bytes_of(1, N, 2)},
                   {A, bytes_of(r, K, 2)},
                   {B, bytes_of(N, r, 2)},
                   {R != Y ? R : nullptr, bytes_of(M, N, 2)}}) ||
      any_overlap({ws}, {{R, bytes_of(M, N, 2)}}))
    return LYNX_ERR_INVALID_ARG;
  const int sms = device_sm_count();
  if (sms == 0) return LYNX_ERR_CUDA;
  LinearW4Launch p;
  std::memset(&p, 0, sizeof(p));
  p.x = X;
  p.wq = Wq;
  p.scales = scales;
  p.zeros = zeros;
  p.bias = bias;
  p.a = A;
  p.b = B;
  p.t = static_cast<float*>(workspace);
  p.y = Y;
  p.N = N;
  p.K = K;
  p.M = static_cast<int>(M);
  p.r = A != nullptr ? static_cast<int>(r) : 0;
  p.group = group;
  p.act = act;
  p.residual = R;
  return status_of(launch_linear_w4(p, sms, static_cast<cudaStream_t>(stream)));
}

size_t lynx_ckpt8_exponent_bytes(int64_t M, int64_t K) {
  if (M <= 0 || K <= 0) return 0;
  return static_cast<size_t>(M) * static_cast<size_t>(K) / 32;
}

int lynx_ckpt8_store(const void* X, int64_t M, int64_t K, int format, void* q, void* e, void* stream) {
  if (any_null(X, q, e) || !format_ok(format)) return LYNX_ERR_INVALID_ARG;
  if (!rows_ok(M) || !k_ok(K)) return LYNX_ERR_UNSUPPORTED_SHAPE;
  if (any_misaligned(X, q, e)) return LYNX_ERR_MISALIGNED;
  if (any_overlap({{q, bytes_of(M, K, 1)}, {e, bytes_of(M, K / 32, 1)}}, {{X, bytes_of(M, K, 2)}}))
    return LYNX_ERR_INVALID_ARG;
  const int sms = device_sm_count();
  if (sms == 0) return LYNX_ERR_CUDA;
  return status_of(launch_ckpt8_store(X, q, e, M * K, format, sms, static_cast<cudaStream_t>(stream)));
}

int lynx_ckpt8_restore(const void* q, const void* e, int64_t M, int64_t K, int format, void* X, void* stream) {
  if (any_null(X, q, e) || !format_ok(format)) return LYNX_ERR_INVALID_ARG;
  if (!rows_ok(M) || !k_ok(K)) return LYNX_ERR_UNSUPPORTED_SHAPE;
  if (any_misaligned(X, q, e)) return LYNX_ERR_MISALIGNED;
  if (any_overlap({{X, bytes_of(M, K, 2)}}, {{q, bytes_of(M, K, 1)}, {e, bytes_of(M, K / 32, 1)}}))
    return LYNX_ERR_INVALID_ARG;
  const int sms = device_sm_count();
  if (sms == 0) return LYNX_ERR_CUDA;
  return status_of(launch_ckpt8_restore(q, e, X, M * K, format, sms, static_cast<cudaStream_t>(stream)));
}

size_t lynx_lora_backward_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t r) {
  if (!rows_ok(M) || !n_ok(N) || !k_ok(K) || !rank_ok(r)) return 0;
  return align256(lora_backward_workspace(M, N, K, r));
}

int lynx_lora_backward(const void* dY, const void* q, const void* e, const void* A, const void* B, int64_t M,
                       int64_t N, int64_t K, int64_t r, int format, void* dA, void* dB, void* dT, void* workspace,
                       size_t workspace_bytes, void* stream) {
  if (any_null(dY, q, e, A, B, dA, dB) || !format_ok(format)) return LYNX_ERR_INVALID_ARG;
  if (!rows_ok(M) || !n_ok(N) || !k_ok(K) || !rank_ok(r)) return LYNX_ERR_UNSUPPORTED_SHAPE;
  if (any_misaligned(dY, q, e, A, B, dA, dB, dT, workspace)) return LYNX_ERR_MISALIGNED;
  if (workspace == nullptr) return LYNX_ERR_INVALID_ARG;
  const size_t need = lynx_lora_backward_workspace_bytes(M, N, K, r);
  if (workspace_bytes < need) return LYNX_ERR_WORKSPACE_TOO_SMALL;
  if (any_overlap({{dA, bytes_of(r, K, 2)}, {dB, bytes_of(N, r, 2)}, {dT, bytes_of(M, r, 2)}, {workspace, need}},
                  {{dY, bytes_of(M, N, 2)},
                   {q, bytes_of(M, K, 1)},
                   {e, bytes_of(M, K / 32, 1)},
                   {A, bytes_of(r, K, 2)},
                   {B, bytes_of(N, r, 2)}}))
    return LYNX_ERR_INVALID_ARG;
  uint32_t* status = stream_status_word(static_cast<cudaStream_t>(stream));
  if (status == nullptr) return LYNX_ERR_CUDA;
  LoraBackwardLaunch p;
  std::memset(&p, 0, sizeof(p));
  p.dy = dY;
  p.q = q;
  p.e = e;
  p.a = A;
  p.b = B;
  p.da = dA;
  p.db = dB;
  p.dt = dT;
  p.ws = static_cast<uint8_t*>(workspace);
  p.M = M;
  p.N = N;
  p.K = K;
  p.r = static_cast<int>(r);
  p.format = format;
  p.stall_test = stall_test_enabled();
  p.status = status;
  return status_of(launch_lora_backward(p, static_cast<cudaStream_t>(stream)));
}

size_t lynx_sparsify_backward_workspace_bytes(int64_t M, int64_t K) {
  if (!rows_ok(M) || !k_ok(K)) return 0;
  return align256(static_cast<size_t>(M) * sizeof(float2));
}

}  // extern "C"

namespace {

// meta null: the selection of the checkpoint's values
int sparsify_backward(const void* G, const void* q, const void* e, const void* meta, const void* dT, const void* A,
                      int64_t M, int64_t K, int64_t r, int format, void* dX, void* workspace, size_t workspace_bytes,
                      void* stream) {
  if (any_null(G, q, e, dX) || !format_ok(format)) return LYNX_ERR_INVALID_ARG;
  if (const int st = check_branch(dT, A, r)) return st;
  if (!rows_ok(M) || !k_ok(K)) return LYNX_ERR_UNSUPPORTED_SHAPE;
  if (any_misaligned(G, q, e, meta, dT, A, dX, workspace)) return LYNX_ERR_MISALIGNED;
  if (workspace == nullptr) return LYNX_ERR_INVALID_ARG;
  const size_t need = lynx_sparsify_backward_workspace_bytes(M, K);
  if (workspace_bytes < need) return LYNX_ERR_WORKSPACE_TOO_SMALL;
  if (any_overlap({{dX, bytes_of(M, K, 2)}, {workspace, need}}, {{G, bytes_of(M, K, 2)},
                                                                 {q, bytes_of(M, K, 1)},
                                                                 {e, bytes_of(M, K / 32, 1)},
                                                                 {meta, lynx_meta_bytes(M, K)},
                                                                 {dT, bytes_of(M, r, 2)},
                                                                 {A, bytes_of(r, K, 2)}}))
    return LYNX_ERR_INVALID_ARG;
  const int sms = device_sm_count();
  uint32_t* status = stream_status_word(static_cast<cudaStream_t>(stream));
  if (sms == 0 || status == nullptr) return LYNX_ERR_CUDA;
  SparsifyBackwardLaunch p;
  std::memset(&p, 0, sizeof(p));
  p.g = G;
  p.q = q;
  p.e = e;
  p.dt = dT;
  p.a = A;
  p.meta = meta;
  p.dx = dX;
  p.coef = static_cast<float2*>(workspace);
  p.M = M;
  p.K = K;
  p.r = dT != nullptr ? static_cast<int>(r) : 0;
  p.format = format;
  p.stall_test = stall_test_enabled();
  p.status = status;
  return status_of(launch_sparsify_backward(p, sms, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

int lynx_sparsify_backward(const void* G, const void* q, const void* e, const void* dT, const void* A, int64_t M,
                           int64_t K, int64_t r, int format, void* dX, void* workspace, size_t workspace_bytes,
                           void* stream) {
  return sparsify_backward(G, q, e, nullptr, dT, A, M, K, r, format, dX, workspace, workspace_bytes, stream);
}

int lynx_sparsify_backward_meta(const void* G, const void* q, const void* e, const void* meta, const void* dT,
                                const void* A, int64_t M, int64_t K, int64_t r, int format, void* dX, void* workspace,
                                size_t workspace_bytes, void* stream) {
  if (meta == nullptr) return LYNX_ERR_INVALID_ARG;
  return sparsify_backward(G, q, e, meta, dT, A, M, K, r, format, dX, workspace, workspace_bytes, stream);
}

// ---- layer norm, the activation's backward pass

int64_t lynx_layer_norm_max_cols(void) { return LYNX_LAYER_NORM_MAX_COLS; }

int lynx_layer_norm(const void* X, const void* weight, const void* bias, int64_t M, int64_t K, float eps, void* Y,
                    float* mean, float* rstd, void* stream) {
  static_assert(kLayerNormMaxCols == LYNX_LAYER_NORM_MAX_COLS, "");
  if (any_null(X, Y) || (mean == nullptr) != (rstd == nullptr) || !eps_ok(eps)) return LYNX_ERR_INVALID_ARG;
  if (!rows_ok(M) || !norm_cols_ok(K)) return LYNX_ERR_UNSUPPORTED_SHAPE;
  if (any_misaligned(X, weight, bias, Y, mean, rstd)) return LYNX_ERR_MISALIGNED;
  if (any_overlap({{Y, bytes_of(M, K, 2)}, {mean, bytes_of(M, 1, 4)}, {rstd, bytes_of(M, 1, 4)}},
                  {{X, bytes_of(M, K, 2)}, {weight, bytes_of(1, K, 2)}, {bias, bytes_of(1, K, 2)}}))
    return LYNX_ERR_INVALID_ARG;
  const int sms = device_sm_count();
  if (sms == 0) return LYNX_ERR_CUDA;
  LayerNormLaunch p = {};
  p.x = X;
  p.w = weight;
  p.b = bias;
  p.y = Y;
  p.mean = mean;
  p.rstd = rstd;
  p.M = M;
  p.K = K;
  p.eps = eps;
  return status_of(launch_layer_norm(p, sms, static_cast<cudaStream_t>(stream)));
}

size_t lynx_layer_norm_backward_workspace_bytes(int64_t M, int64_t K) {
  if (!rows_ok(M) || !norm_cols_ok(K)) return 0;
  return align256(layer_norm_backward_workspace(M, K));
}

int lynx_layer_norm_backward(const void* dY, const void* X, const float* mean, const float* rstd, const void* weight,
                             const void* dR, int64_t M, int64_t K, void* dX, void* dweight, void* dbias, void* workspace,
                             size_t workspace_bytes, void* stream) {
  if (any_null(dY, X, mean, rstd, dX)) return LYNX_ERR_INVALID_ARG;
  if (!rows_ok(M) || !norm_cols_ok(K)) return LYNX_ERR_UNSUPPORTED_SHAPE;
  if (any_misaligned(dY, X, mean, rstd, weight, dR, dX, dweight, dbias, workspace)) return LYNX_ERR_MISALIGNED;
  const bool sums = dweight != nullptr || dbias != nullptr;
  const size_t need = sums ? lynx_layer_norm_backward_workspace_bytes(M, K) : 0;
  if (need != 0 && workspace == nullptr) return LYNX_ERR_INVALID_ARG;
  if (workspace_bytes < need) return LYNX_ERR_WORKSPACE_TOO_SMALL;
  const Span ws = {need != 0 ? workspace : nullptr, need}, dw = {dweight, bytes_of(1, K, 2)}, db = {dbias, bytes_of(1, K, 2)};
  if (any_overlap({{dX, bytes_of(M, K, 2)}, dw, db, ws},
                  {{dY, bytes_of(M, K, 2)},
                   {X, bytes_of(M, K, 2)},
                   {mean, bytes_of(M, 1, 4)},
                   {rstd, bytes_of(M, 1, 4)},
                   {weight, bytes_of(1, K, 2)},
                   {dR != dX ? dR : nullptr, bytes_of(M, K, 2)}}) ||
      any_overlap({dw, db, ws}, {{dR, bytes_of(M, K, 2)}}))
    return LYNX_ERR_INVALID_ARG;
  if (device_sm_count() == 0) return LYNX_ERR_CUDA;
  LayerNormBackwardLaunch p = {};
  p.dy = dY;
  p.x = X;
  p.w = weight;
  p.mean = mean;
  p.rstd = rstd;
  p.dr = dR;
  p.dx = dX;
  p.dw = dweight;
  p.db = dbias;
  p.part = need != 0 ? static_cast<float*>(workspace) : nullptr;
  p.M = M;
  p.K = K;
  return status_of(launch_layer_norm_backward(p, static_cast<cudaStream_t>(stream)));
}

size_t lynx_act_backward_workspace_bytes(int64_t M, int64_t N) {
  if (!rows_ok(M) || !n_ok(N)) return 0;
  return align256(column_pass_workspace(M, N, 1));
}

int lynx_act_backward(const void* dY, const void* Z, int64_t M, int64_t N, int act, void* dZ, void* dbias,
                      void* workspace, size_t workspace_bytes, void* stream) {
  if (act != LYNX_ACT_NONE && act != LYNX_ACT_GELU_TANH) return LYNX_ERR_INVALID_ARG;
  if (dY == nullptr) return LYNX_ERR_INVALID_ARG;
  if (act == LYNX_ACT_NONE ? Z != nullptr || dZ != nullptr || dbias == nullptr : any_null(Z, dZ))
    return LYNX_ERR_INVALID_ARG;
  if (!rows_ok(M) || !n_ok(N)) return LYNX_ERR_UNSUPPORTED_SHAPE;
  if (any_misaligned(dY, Z, dZ, dbias, workspace)) return LYNX_ERR_MISALIGNED;
  const size_t need = dbias != nullptr ? lynx_act_backward_workspace_bytes(M, N) : 0;
  if (need != 0 && workspace == nullptr) return LYNX_ERR_INVALID_ARG;
  if (workspace_bytes < need) return LYNX_ERR_WORKSPACE_TOO_SMALL;
  const Span ws = {need != 0 ? workspace : nullptr, need}, db = {dbias, bytes_of(1, N, 2)};
  const Span dy = {dY, bytes_of(M, N, 2)}, z = {Z, bytes_of(M, N, 2)};
  if (any_overlap({{dZ, bytes_of(M, N, 2)}, db, ws}, {z}) || any_overlap({db, ws}, {dy}) ||
      (dZ != dY && any_overlap({{dZ, bytes_of(M, N, 2)}}, {dy})))
    return LYNX_ERR_INVALID_ARG;
  if (device_sm_count() == 0) return LYNX_ERR_CUDA;
  ColumnPassLaunch p = {};
  p.dy = dY;
  p.z = Z;
  p.dz = dZ;
  p.out0 = dbias;
  p.part = need != 0 ? static_cast<float*>(workspace) : nullptr;
  p.M = M;
  p.N = N;
  return status_of(launch_act_backward(p, act, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
