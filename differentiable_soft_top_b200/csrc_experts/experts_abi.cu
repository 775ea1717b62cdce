// experts_abi.cu -- the C ABI of lapsum_experts.h: argument checks and the
// choice of launches.
#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "experts.h"

namespace lapsum {
namespace {

constexpr int kMaxDevices = 64;
struct DevInfo {
  std::atomic<bool> ready{false};
  int sms = 0;
};
DevInfo g_dev[kMaxDevices];
std::mutex g_mu;
thread_local const char* t_error = "no error";

bool cuda_ok(cudaError_t e) {
  if (e == cudaSuccess) return true;
  t_error = cudaGetErrorString(e);
  return false;
}
int done(cudaError_t e) { return cuda_ok(e) ? LAPSUM_OK : LAPSUM_ECUDA; }

// the current device's SM count; 0 after a CUDA error
int device_sms() {
  int dev = 0;
  if (!cuda_ok(cudaGetDevice(&dev))) return 0;
  if (dev < 0 || dev >= kMaxDevices) {
    t_error = "device number out of range";
    return 0;
  }
  // tensor maps are encoded by the driver, which wants the device's context
  // current on this host thread (a thread that has launched nothing has none)
  thread_local int t_dev = -1;
  if (t_dev != dev) {
    if (!cuda_ok(cudaSetDevice(dev))) return 0;
    t_dev = dev;
  }
  DevInfo& d = g_dev[dev];
  if (!d.ready.load(std::memory_order_acquire)) {
    std::lock_guard<std::mutex> lk(g_mu);
    if (!d.ready.load(std::memory_order_relaxed)) {
      if (!cuda_ok(cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev))) return 0;
      if (!cuda_ok(linear_init_bf16()) || !cuda_ok(linear_init_f16()) || !cuda_ok(exchange_init())) return 0;
      d.ready.store(true, std::memory_order_release);
    }
  }
  return d.sms;
}

bool overlaps(const void* a, size_t an, const void* b, size_t bn) {
  if (!a || !b) return false;
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + bn && y < x + an;
}
size_t span(int64_t rows, int64_t cols, int64_t stride, int size) {
  return rows < 1 ? 0 : (size_t)((rows - 1) * stride + cols) * size;
}
bool aligned(const void* p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) == 0; }
bool known(int dtype) { return dtype == LAPSUM_F32 || dtype == LAPSUM_BF16 || dtype == LAPSUM_F16; }
int size_of(int dtype) { return dtype == LAPSUM_F32 ? 4 : 2; }
constexpr int64_t kMaxIndex = INT32_MAX;

// polls of a product's bounded waits (2^20: about a second), and the test knob
constexpr uint32_t kPolls = 1u << 20;
thread_local uint32_t t_test_polls = 0;
void set_limits(Product& p) {
  p.polls = t_test_polls ? t_test_polls : kPolls;
  p.starve = t_test_polls != 0;
}

// A 16-bit matrix that tiled copies and 16-byte accesses reach: 16-byte rows.
bool matrix16(const void* p, int64_t cols, int64_t stride) {
  return p && aligned(p, 16) && stride >= cols && stride % 8 == 0 && stride < (int64_t(1) << 37);
}
bool experts_shape(int experts, const int32_t* offsets) {
  return experts >= 1 && experts <= LAPSUM_EXPERTS_MAX && aligned(offsets, 4) && (offsets || experts == 1);
}
// rows leave room for a tile behind the last one in 32-bit coordinates
bool linear_shape(int dtype, int64_t rows, int64_t in, int64_t out) {
  return (dtype == LAPSUM_BF16 || dtype == LAPSUM_F16) && rows >= 1 && rows <= kMaxIndex - 1024 && in >= 8 && out >= 8 &&
         in % 8 == 0 && out % 8 == 0 && in <= (1 << 24) && out <= (1 << 24);
}
// tiles are counted in 32 bits
bool tiles_fit(int64_t rows, int experts, int64_t in, int64_t out) {
  const int64_t f = (std::max(in, out) + 127) / 128;
  return (experts + 1 + rows / 32) * f * 8 <= kMaxIndex && (int64_t)experts * f * f <= kMaxIndex;
}

}  // namespace
}  // namespace lapsum

using namespace lapsum;

extern "C" {

const char* lapsum_experts_last_cuda_error(void) { return t_error; }

void lapsum_experts_test_timeout(uint32_t polls) { t_test_polls = polls; }

static int route_args(const void* scores, int dtype, int64_t tokens, int experts, int64_t row_stride, int k, int score,
                      const float* bias, float scale) {
  if (!scores || !known(dtype) || tokens < 1 || experts < 1 || row_stride < experts) return LAPSUM_EINVAL;
  if (experts > LAPSUM_EXPERTS_MAX || k > LAPSUM_EXPERTS_MAX_K || tokens > kMaxIndex / LAPSUM_EXPERTS_MAX_K)
    return LAPSUM_ETOOLARGE;
  if (!aligned(scores, size_of(dtype)) || !aligned(bias, 4)) return LAPSUM_EINVAL;
  if (score != LAPSUM_SCORE_SOFTMAX && score != LAPSUM_SCORE_SIGMOID && score != LAPSUM_SCORE_IDENTITY)
    return LAPSUM_EINVAL;
  if (k < 1 || k > experts) return LAPSUM_EBADK;
  if (!std::isfinite(scale) || !(scale > 0.0f)) return LAPSUM_EINVAL;
  return LAPSUM_OK;
}

int lapsum_experts_route_fwd(const void* scores, int dtype, int64_t tokens, int experts, int64_t row_stride, int k,
                             int score, const float* bias, int groups, int groups_kept, int group_top, int renormalize,
                             float scale, float* weights, int32_t* chosen, void* stream) {
  const int rc = route_args(scores, dtype, tokens, experts, row_stride, k, score, bias, scale);
  if (rc != LAPSUM_OK) return rc;
  if (!weights || !chosen || !aligned(weights, 4) || !aligned(chosen, 4)) return LAPSUM_EINVAL;
  if (groups < 1 || groups > LAPSUM_EXPERTS_MAX_GROUPS || experts % groups || groups_kept < 1 || groups_kept > groups)
    return LAPSUM_EINVAL;
  if (group_top != 1 && group_top != 2) return LAPSUM_EINVAL;
  if (k > experts / groups * groups_kept) return LAPSUM_EBADK;
  const size_t in = span(tokens, experts, row_stride, size_of(dtype)), out = 4 * (size_t)tokens * k;
  if (overlaps(scores, in, weights, out) || overlaps(scores, in, chosen, out) || overlaps(weights, out, chosen, out) ||
      overlaps(bias, 4 * (size_t)experts, weights, out) || overlaps(bias, 4 * (size_t)experts, chosen, out))
    return LAPSUM_EINVAL;
  if (!device_sms()) return LAPSUM_ECUDA;
  RouteFwd a{scores, dtype, tokens, row_stride, experts, k, score, bias, groups, groups_kept, group_top,
             renormalize != 0, scale, weights, chosen, false, false};
  return done(launch_route_fwd(a, (cudaStream_t)stream));
}

int lapsum_experts_route_bwd(const void* scores, int dtype, int64_t tokens, int experts, int64_t row_stride, int k,
                             int score, const float* bias, int renormalize, float scale, const int32_t* chosen,
                             const float* weights, const float* grad_weights, void* grad_scores, int64_t grad_stride,
                             void* stream) {
  const int rc = route_args(scores, dtype, tokens, experts, row_stride, k, score, bias, scale);
  if (rc != LAPSUM_OK) return rc;
  if (!chosen || !weights || !grad_weights || !grad_scores || grad_stride < experts) return LAPSUM_EINVAL;
  if (!aligned(chosen, 4) || !aligned(weights, 4) || !aligned(grad_weights, 4) ||
      !aligned(grad_scores, size_of(dtype)))
    return LAPSUM_EINVAL;
  const size_t out = span(tokens, experts, grad_stride, size_of(dtype)), small = 4 * (size_t)tokens * k;
  if (overlaps(scores, span(tokens, experts, row_stride, size_of(dtype)), grad_scores, out) ||
      overlaps(chosen, small, grad_scores, out) || overlaps(weights, small, grad_scores, out) ||
      overlaps(grad_weights, small, grad_scores, out) || overlaps(bias, 4 * (size_t)experts, grad_scores, out))
    return LAPSUM_EINVAL;
  if (!device_sms()) return LAPSUM_ECUDA;
  RouteBwd a{scores, dtype, tokens, row_stride, experts, k, score, bias, renormalize != 0, scale, chosen, weights,
             grad_weights, grad_scores, grad_stride, false, false, false};
  return done(launch_route_bwd(a, (cudaStream_t)stream));
}

size_t lapsum_experts_plan_workspace_size(int64_t slots, int experts) {
  if (slots < 1 || slots > kMaxIndex || experts < 1 || experts > LAPSUM_EXPERTS_MAX) return 0;
  return plan_workspace(slots, experts);
}

int lapsum_experts_plan(const int32_t* chosen, int64_t slots, int experts, int32_t* offsets, int32_t* rows,
                        int32_t* slot_of, void* workspace, size_t workspace_bytes, void* stream) {
  if (!chosen || !offsets || !rows || !slot_of || slots < 1 || experts < 1) return LAPSUM_EINVAL;
  if (slots > kMaxIndex || experts > LAPSUM_EXPERTS_MAX) return LAPSUM_ETOOLARGE;
  if (!aligned(chosen, 4) || !aligned(offsets, 4) || !aligned(rows, 4) || !aligned(slot_of, 4)) return LAPSUM_EINVAL;
  const size_t n = 4 * (size_t)slots, o = 4 * (size_t)(experts + 1);
  if (overlaps(chosen, n, offsets, o) || overlaps(chosen, n, rows, n) || overlaps(chosen, n, slot_of, n) ||
      overlaps(rows, n, slot_of, n) || overlaps(rows, n, offsets, o) || overlaps(slot_of, n, offsets, o))
    return LAPSUM_EINVAL;
  const size_t need = plan_workspace(slots, experts);
  if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 256))) return LAPSUM_EWORKSPACE;
  if (!device_sms()) return LAPSUM_ECUDA;
  return done(launch_plan(chosen, slots, experts, offsets, rows, slot_of, workspace, (cudaStream_t)stream));
}

static int rows_args(int dtype, int64_t tokens, int k, int64_t dim) {
  if (!known(dtype) || tokens < 1 || k < 1 || dim < 1) return LAPSUM_EINVAL;
  if (k > LAPSUM_EXPERTS_MAX_K || tokens > kMaxIndex / k || dim > (1 << 24)) return LAPSUM_ETOOLARGE;
  return LAPSUM_OK;
}

int lapsum_experts_dispatch(const void* x, int dtype, int64_t tokens, int k, int64_t dim, int64_t x_stride,
                            const int32_t* slot_of, void* out, int64_t out_stride, void* stream) {
  const int rc = rows_args(dtype, tokens, k, dim);
  if (rc != LAPSUM_OK) return rc;
  const int z = size_of(dtype);
  if (!x || !slot_of || !out || x_stride < dim || out_stride < dim) return LAPSUM_EINVAL;
  if (!aligned(x, z) || !aligned(out, z) || !aligned(slot_of, 4)) return LAPSUM_EINVAL;
  const size_t o = span(tokens * k, dim, out_stride, z);
  if (overlaps(x, span(tokens, dim, x_stride, z), out, o) || overlaps(slot_of, 4 * (size_t)(tokens * k), out, o))
    return LAPSUM_EINVAL;
  const int sms = device_sms();
  if (!sms) return LAPSUM_ECUDA;
  return done(launch_dispatch(x, dtype, tokens, k, dim, x_stride, slot_of, out, out_stride, sms, (cudaStream_t)stream));
}

int lapsum_experts_combine(const void* y, int dtype, int64_t tokens, int k, int64_t dim, int64_t y_stride,
                           const float* weights, const int32_t* rows, const void* residual, int64_t residual_stride,
                           void* out, int64_t out_stride, void* stream) {
  const int rc = rows_args(dtype, tokens, k, dim);
  if (rc != LAPSUM_OK) return rc;
  const int z = size_of(dtype);
  if (!y || !rows || !out || y_stride < dim || out_stride < dim || (residual && residual_stride < dim))
    return LAPSUM_EINVAL;
  if (!aligned(y, z) || !aligned(out, z) || !aligned(residual, z) || !aligned(weights, 4) || !aligned(rows, 4))
    return LAPSUM_EINVAL;
  const size_t o = span(tokens, dim, out_stride, z), n = 4 * (size_t)(tokens * k);
  if (overlaps(y, span(tokens * k, dim, y_stride, z), out, o) || overlaps(weights, n, out, o) ||
      overlaps(rows, n, out, o) || overlaps(residual, span(tokens, dim, residual_stride, z), out, o))
    return LAPSUM_EINVAL;
  const int sms = device_sms();
  if (!sms) return LAPSUM_ECUDA;
  return done(launch_combine(y, dtype, tokens, k, dim, y_stride, weights, rows, residual, residual_stride, out,
                             out_stride, sms, (cudaStream_t)stream));
}

int lapsum_experts_combine_bwd(const void* grad, int dtype, int64_t tokens, int k, int64_t dim, int64_t grad_stride,
                               const void* y, int64_t y_stride, const float* weights, const int32_t* rows,
                               const int32_t* slot_of, void* grad_y, int64_t grad_y_stride, float* grad_weights,
                               void* stream) {
  const int rc = rows_args(dtype, tokens, k, dim);
  if (rc != LAPSUM_OK) return rc;
  const int z = size_of(dtype);
  if (!grad || !rows || !slot_of || grad_stride < dim || (!grad_y && !grad_weights)) return LAPSUM_EINVAL;
  if ((grad_weights && (!y || y_stride < dim)) || (grad_y && grad_y_stride < dim)) return LAPSUM_EINVAL;
  if (!aligned(grad, z) || !aligned(y, z) || !aligned(grad_y, z) || !aligned(weights, 4) || !aligned(rows, 4) ||
      !aligned(slot_of, 4) || !aligned(grad_weights, 4))
    return LAPSUM_EINVAL;
  const size_t go = span(tokens, dim, grad_stride, z), yo = span(tokens * k, dim, y_stride, z), n = 4 * (size_t)(tokens * k);
  struct {
    const void* p;
    size_t n;
  } outs[2] = {{grad_y, span(tokens * k, dim, grad_y_stride, z)}, {grad_weights, n}},
    ins[5] = {{grad, go}, {y, yo}, {weights, n}, {rows, n}, {slot_of, n}};
  for (const auto& o : outs)
    for (const auto& i : ins)
      if (overlaps(o.p, o.n, i.p, i.n)) return LAPSUM_EINVAL;
  if (overlaps(outs[0].p, outs[0].n, outs[1].p, outs[1].n)) return LAPSUM_EINVAL;
  const int sms = device_sms();
  if (!sms) return LAPSUM_ECUDA;
  return done(launch_combine_bwd(grad, dtype, tokens, k, dim, grad_stride, y, y_stride, weights, rows, slot_of, grad_y,
                                 grad_y_stride, grad_weights, sms, (cudaStream_t)stream));
}

int lapsum_experts_linear_fwd(const void* x, int dtype, int64_t rows, int64_t in, int64_t x_stride, const void* weight,
                              int experts, int64_t out, const int32_t* offsets, const void* bias, int activation,
                              const void* residual, int64_t residual_stride, void* y, int64_t y_stride, void* preact,
                              int64_t preact_stride, uint32_t* status, void* stream) {
  if (!linear_shape(dtype, rows, in, out) || !experts_shape(experts, offsets)) return LAPSUM_EINVAL;
  if (activation < LAPSUM_ACT_NONE || activation > LAPSUM_ACT_SWIGLU) return LAPSUM_EINVAL;
  const bool gated = activation == LAPSUM_ACT_SWIGLU;
  if (gated && out % 16) return LAPSUM_EINVAL;
  if (!tiles_fit(rows, experts, in, out)) return LAPSUM_ETOOLARGE;
  const int64_t width = gated ? out / 2 : out;
  if (!matrix16(x, in, x_stride) || !weight || !aligned(weight, 16) || !matrix16(y, width, y_stride)) return LAPSUM_EINVAL;
  if ((residual && !matrix16(residual, width, residual_stride)) || (preact && !matrix16(preact, out, preact_stride)) ||
      !aligned(bias, 2) || !aligned(status, 4))
    return LAPSUM_EINVAL;
  struct {
    const void* p;
    size_t n;
  } outs[2] = {{y, span(rows, width, y_stride, 2)}, {preact, span(rows, out, preact_stride, 2)}},
    ins[5] = {{x, span(rows, in, x_stride, 2)},
              {weight, 2 * (size_t)experts * out * in},
              {bias, 2 * (size_t)experts * out},
              {residual, span(rows, width, residual_stride, 2)},
              {offsets, 4 * (size_t)(experts + 1)}};
  for (const auto& o : outs)
    for (const auto& i : ins)
      if (overlaps(o.p, o.n, i.p, i.n)) return LAPSUM_EINVAL;
  if (overlaps(outs[0].p, outs[0].n, outs[1].p, outs[1].n)) return LAPSUM_EINVAL;
  const int sms = device_sms();
  if (!sms) return LAPSUM_ECUDA;
  Product p{};
  p.rows = rows;
  p.experts = experts;
  p.activation = activation;
  p.in = in;
  p.out = out;
  p.offsets = offsets;
  p.x = x;
  p.x_stride = x_stride;
  p.weight = weight;
  p.bias = bias;
  p.residual = residual;
  p.residual_stride = residual_stride;
  p.y = y;
  p.y_stride = y_stride;
  p.preact = preact;
  p.preact_stride = preact_stride;
  p.status = status;
  set_limits(p);
  return done((dtype == LAPSUM_BF16 ? launch_linear_fwd_bf16 : launch_linear_fwd_f16)(p, sms, (cudaStream_t)stream));
}

size_t lapsum_experts_linear_act_workspace_size(int64_t rows, int experts, int64_t out) {
  if (rows < 1 || experts < 1 || experts > LAPSUM_EXPERTS_MAX || out < 1) return 0;
  return act_bwd_workspace(rows, experts, out);
}

int lapsum_experts_linear_act_bwd(const void* grad_y, int dtype, int64_t rows, int64_t out, int64_t grad_y_stride,
                                  const void* preact, int64_t preact_stride, int experts, const int32_t* offsets,
                                  int activation, void* grad_h, int64_t grad_h_stride, void* grad_bias,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  if (!linear_shape(dtype, rows, 8, out) || !experts_shape(experts, offsets)) return LAPSUM_EINVAL;
  if (activation < LAPSUM_ACT_NONE || activation > LAPSUM_ACT_SWIGLU) return LAPSUM_EINVAL;
  const bool gated = activation == LAPSUM_ACT_SWIGLU, plain = activation == LAPSUM_ACT_NONE;
  if (gated && out % 16) return LAPSUM_EINVAL;
  if (!tiles_fit(rows, experts, 8, out)) return LAPSUM_ETOOLARGE;
  const int64_t width = gated ? out / 2 : out;
  if (!matrix16(grad_y, width, grad_y_stride) || !aligned(grad_bias, 2)) return LAPSUM_EINVAL;
  if (!plain && (!matrix16(preact, out, preact_stride) || !grad_h)) return LAPSUM_EINVAL;
  if (grad_h ? !matrix16(grad_h, out, grad_h_stride) : !grad_bias) return LAPSUM_EINVAL;
  const size_t need = grad_bias ? act_bwd_workspace(rows, experts, out) : 0;
  if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 256))) return LAPSUM_EWORKSPACE;
  struct {
    const void* p;
    size_t n;
  } outs[3] = {{grad_h, span(rows, out, grad_h_stride, 2)}, {grad_bias, 2 * (size_t)experts * out}, {workspace, need}},
    ins[3] = {{grad_y, span(rows, width, grad_y_stride, 2)},
              {plain ? nullptr : preact, span(rows, out, preact_stride, 2)},
              {offsets, 4 * (size_t)(experts + 1)}};
  for (const auto& o : outs)
    for (const auto& i : ins)
      if (overlaps(o.p, o.n, i.p, i.n)) return LAPSUM_EINVAL;
  for (int i = 0; i < 3; ++i)
    if (overlaps(outs[i].p, outs[i].n, outs[(i + 1) % 3].p, outs[(i + 1) % 3].n)) return LAPSUM_EINVAL;
  const int sms = device_sms();
  if (!sms) return LAPSUM_ECUDA;
  return done(launch_act_bwd(grad_y, dtype == LAPSUM_BF16, rows, out, grad_y_stride, preact, preact_stride, experts,
                             offsets, activation, grad_h, grad_h_stride, grad_bias, workspace, sms,
                             (cudaStream_t)stream));
}

int lapsum_experts_linear_dx(const void* grad_h, int dtype, int64_t rows, int64_t out, int64_t grad_h_stride,
                             const void* weight, int experts, int64_t in, const int32_t* offsets, void* grad_x,
                             int64_t grad_x_stride, uint32_t* status, void* stream) {
  if (!linear_shape(dtype, rows, in, out) || !experts_shape(experts, offsets)) return LAPSUM_EINVAL;
  if (!tiles_fit(rows, experts, in, out)) return LAPSUM_ETOOLARGE;
  if (!matrix16(grad_h, out, grad_h_stride) || !weight || !aligned(weight, 16) || !matrix16(grad_x, in, grad_x_stride) ||
      !aligned(status, 4))
    return LAPSUM_EINVAL;
  const size_t o = span(rows, in, grad_x_stride, 2);
  if (overlaps(grad_x, o, grad_h, span(rows, out, grad_h_stride, 2)) ||
      overlaps(grad_x, o, weight, 2 * (size_t)experts * out * in) ||
      overlaps(grad_x, o, offsets, 4 * (size_t)(experts + 1)))
    return LAPSUM_EINVAL;
  const int sms = device_sms();
  if (!sms) return LAPSUM_ECUDA;
  Product p{};
  p.rows = rows;
  p.experts = experts;
  p.in = in;
  p.out = out;
  p.offsets = offsets;
  p.grad_h = grad_h;
  p.grad_h_stride = grad_h_stride;
  p.weight = weight;
  p.y = grad_x;
  p.y_stride = grad_x_stride;
  p.status = status;
  set_limits(p);
  return done((dtype == LAPSUM_BF16 ? launch_linear_dx_bf16 : launch_linear_dx_f16)(p, sms, (cudaStream_t)stream));
}

int lapsum_experts_linear_dweight(const void* grad_h, int dtype, int64_t rows, int64_t out, int64_t grad_h_stride,
                                  const void* x, int64_t in, int64_t x_stride, int experts, const int32_t* offsets,
                                  void* grad_weight, uint32_t* status, void* stream) {
  if (!linear_shape(dtype, rows, in, out) || !experts_shape(experts, offsets)) return LAPSUM_EINVAL;
  if (!tiles_fit(rows, experts, in, out)) return LAPSUM_ETOOLARGE;
  if (!matrix16(grad_h, out, grad_h_stride) || !matrix16(x, in, x_stride) || !grad_weight || !aligned(grad_weight, 16) ||
      !aligned(status, 4))
    return LAPSUM_EINVAL;
  const size_t o = 2 * (size_t)experts * out * in;
  if (overlaps(grad_weight, o, grad_h, span(rows, out, grad_h_stride, 2)) ||
      overlaps(grad_weight, o, x, span(rows, in, x_stride, 2)) ||
      overlaps(grad_weight, o, offsets, 4 * (size_t)(experts + 1)))
    return LAPSUM_EINVAL;
  const int sms = device_sms();
  if (!sms) return LAPSUM_ECUDA;
  Product p{};
  p.rows = rows;
  p.experts = experts;
  p.in = in;
  p.out = out;
  p.offsets = offsets;
  p.x = x;
  p.x_stride = x_stride;
  p.grad_h = grad_h;
  p.grad_h_stride = grad_h_stride;
  p.y = grad_weight;
  p.status = status;
  set_limits(p);
  return done((dtype == LAPSUM_BF16 ? launch_linear_dweight_bf16 : launch_linear_dweight_f16)(p, sms, (cudaStream_t)stream));
}

static size_t round256(size_t n) { return (n + 255) & ~size_t(255); }

size_t lapsum_experts_linear_bwd_workspace_size(int64_t rows, int experts, int64_t out, int activation, int with_bias) {
  if (rows < 1 || experts < 1 || experts > LAPSUM_EXPERTS_MAX || out < 1) return 0;
  return (activation != LAPSUM_ACT_NONE ? round256(2 * (size_t)rows * out) : 0) +
         (with_bias ? act_bwd_workspace(rows, experts, out) : 0);
}

int lapsum_experts_linear_bwd(const void* grad_y, int dtype, int64_t rows, int64_t out, int64_t grad_y_stride,
                              const void* preact, const void* x, int64_t in, int64_t x_stride, const void* weight,
                              int experts, const int32_t* offsets, int activation, void* grad_x, void* grad_weight,
                              void* grad_bias, uint32_t* status, void* workspace, size_t workspace_bytes, void* stream) {
  // everything that a later step could refuse is checked before the first is enqueued
  if (!linear_shape(dtype, rows, in, out) || !experts_shape(experts, offsets)) return LAPSUM_EINVAL;
  if (activation < LAPSUM_ACT_NONE || activation > LAPSUM_ACT_SWIGLU) return LAPSUM_EINVAL;
  const bool gated = activation == LAPSUM_ACT_SWIGLU, plain = activation == LAPSUM_ACT_NONE;
  if (gated && out % 16) return LAPSUM_EINVAL;
  if (!tiles_fit(rows, experts, in, out)) return LAPSUM_ETOOLARGE;
  if (!grad_x && !grad_weight && !grad_bias) return LAPSUM_EINVAL;
  const int64_t width = gated ? out / 2 : out;
  if (!matrix16(grad_y, width, grad_y_stride) || (!plain && !matrix16(preact, out, out)) || !aligned(grad_bias, 2) ||
      !aligned(status, 4))
    return LAPSUM_EINVAL;
  if ((grad_x && (!matrix16(grad_x, in, in) || !weight || !aligned(weight, 16))) ||
      (grad_weight && (!aligned(grad_weight, 16) || !matrix16(x, in, x_stride))))
    return LAPSUM_EINVAL;
  const size_t need = lapsum_experts_linear_bwd_workspace_size(rows, experts, out, activation, grad_bias != nullptr);
  if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 256))) return LAPSUM_EWORKSPACE;
  const size_t wn = 2 * (size_t)experts * out * in;
  struct {
    const void* p;
    size_t n;
  } outs[4] = {{grad_x, span(rows, in, in, 2)}, {grad_weight, wn}, {grad_bias, 2 * (size_t)experts * out}, {workspace, need}},
    ins[5] = {{grad_y, span(rows, width, grad_y_stride, 2)},
              {plain ? nullptr : preact, span(rows, out, out, 2)},
              {grad_weight ? x : nullptr, span(rows, in, x_stride, 2)},
              {grad_x ? weight : nullptr, wn},
              {offsets, 4 * (size_t)(experts + 1)}};
  for (int o = 0; o < 4; ++o) {
    for (const auto& i : ins)
      if (overlaps(outs[o].p, outs[o].n, i.p, i.n)) return LAPSUM_EINVAL;
    for (int q = 0; q < o; ++q)
      if (overlaps(outs[o].p, outs[o].n, outs[q].p, outs[q].n)) return LAPSUM_EINVAL;
  }
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  const size_t gh_bytes = plain ? 0 : round256(2 * (size_t)rows * out);
  const void* gh = plain ? grad_y : ws;
  const int64_t gh_stride = plain ? grad_y_stride : out;
  int rc = LAPSUM_OK;
  if (!plain || grad_bias)
    rc = lapsum_experts_linear_act_bwd(grad_y, dtype, rows, out, grad_y_stride, preact, out, experts, offsets, activation,
                                       plain ? nullptr : ws, out, grad_bias, ws + gh_bytes, workspace_bytes - gh_bytes,
                                       stream);
  if (rc == LAPSUM_OK && grad_x)
    rc = lapsum_experts_linear_dx(gh, dtype, rows, out, gh_stride, weight, experts, in, offsets, grad_x, in, status, stream);
  if (rc == LAPSUM_OK && grad_weight)
    rc = lapsum_experts_linear_dweight(gh, dtype, rows, out, gh_stride, x, in, x_stride, experts, offsets, grad_weight,
                                       status, stream);
  return rc;
}

// Workspace of the layer: the plan's arrays and scratch, then the rows before,
// between and after the products, each on a 256-byte boundary.  The rows are of the
// type: those between the products are the second one's operand, which the tensor
// cores take in 16 bits; those after it (and the pre-activation that is kept) could
// be fp32, for twice the bytes of the layer's largest arrays: a rounding each, half a
// step of the type, as where the products are called one by one.
struct MlpLayout {
  size_t offsets, rows, slots, plan, x_rows, pre, h, y, total;
  int64_t hidden;
};
static MlpLayout mlp_layout(int64_t tokens, int k, int experts, int64_t dim, int64_t up, int activation, int64_t dim_out,
                            bool keep) {
  const size_t n = (size_t)tokens * k;
  MlpLayout l;
  l.hidden = activation == LAPSUM_ACT_SWIGLU ? up / 2 : up;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at = round256(at + bytes);
    return here;
  };
  l.offsets = take(4 * ((size_t)experts + 1));
  l.rows = take(4 * n);
  l.slots = take(4 * n);
  l.plan = take(plan_workspace((int64_t)n, experts));
  l.x_rows = take(2 * n * dim);
  l.pre = take(keep && activation != LAPSUM_ACT_NONE ? 2 * n * up : 0);
  l.h = take(2 * n * l.hidden);
  l.y = take(2 * n * dim_out);
  l.total = at;
  return l;
}
static int mlp_shape(int dtype, int64_t tokens, int k, int experts, int64_t dim, int64_t up, int activation,
                     int64_t dim_out) {
  if (activation < LAPSUM_ACT_NONE || activation > LAPSUM_ACT_SWIGLU) return LAPSUM_EINVAL;
  const bool gated = activation == LAPSUM_ACT_SWIGLU;
  if (tokens < 1 || k < 1 || k > LAPSUM_EXPERTS_MAX_K || tokens > (kMaxIndex - 1024) / k || experts < 1 ||
      experts > LAPSUM_EXPERTS_MAX || up < 1 || (gated && up % 16))
    return LAPSUM_EINVAL;
  const int64_t n = tokens * k, hidden = gated ? up / 2 : up;
  if (!linear_shape(dtype, n, dim, up) || !linear_shape(dtype, n, hidden, dim_out)) return LAPSUM_EINVAL;
  if (!tiles_fit(n, experts, dim, up) || !tiles_fit(n, experts, hidden, dim_out)) return LAPSUM_ETOOLARGE;
  return LAPSUM_OK;
}

size_t lapsum_experts_mlp_workspace_size(int64_t tokens, int k, int experts, int64_t dim, int64_t up, int activation,
                                         int64_t dim_out, int keep) {
  if (mlp_shape(LAPSUM_BF16, tokens, k, experts, dim, up, activation, dim_out) != LAPSUM_OK) return 0;
  return mlp_layout(tokens, k, experts, dim, up, activation, dim_out, keep != 0).total;
}

int lapsum_experts_mlp_fwd(const void* x, int dtype, int64_t tokens, int64_t dim, int64_t x_stride, const float* weights,
                           const int32_t* chosen, int k, const void* w_in, const void* b_in, int experts, int64_t up,
                           int activation, const void* w_out, const void* b_out, int64_t dim_out, const void* residual,
                           int64_t residual_stride, void* out, int64_t out_stride, int keep, uint32_t* status,
                           void* workspace, size_t workspace_bytes, void* stream) {
  // everything that a later step could refuse is checked before the first is enqueued
  int rc = mlp_shape(dtype, tokens, k, experts, dim, up, activation, dim_out);
  if (rc != LAPSUM_OK) return rc;
  const int64_t n = tokens * k;
  if (!x || !weights || !chosen || !w_in || !w_out || !out || x_stride < dim || out_stride < dim_out ||
      (residual && residual_stride < dim_out))
    return LAPSUM_EINVAL;
  if (!aligned(x, 2) || !aligned(out, 2) || !aligned(residual, 2) || !aligned(weights, 4) || !aligned(chosen, 4) ||
      !aligned(w_in, 16) || !aligned(w_out, 16) || !aligned(b_in, 2) || !aligned(b_out, 2) || !aligned(status, 4))
    return LAPSUM_EINVAL;
  const MlpLayout l = mlp_layout(tokens, k, experts, dim, up, activation, dim_out, keep != 0);
  const int64_t hidden = l.hidden;
  if (!workspace || workspace_bytes < l.total || !aligned(workspace, 256)) return LAPSUM_EWORKSPACE;
  struct {
    const void* p;
    size_t n;
  } outs[2] = {{out, span(tokens, dim_out, out_stride, 2)}, {workspace, l.total}},
    ins[8] = {{x, span(tokens, dim, x_stride, 2)},
              {weights, 4 * (size_t)n},
              {chosen, 4 * (size_t)n},
              {w_in, 2 * (size_t)experts * up * dim},
              {b_in, 2 * (size_t)experts * up},
              {w_out, 2 * (size_t)experts * dim_out * hidden},
              {b_out, 2 * (size_t)experts * dim_out},
              {residual, span(tokens, dim_out, residual_stride, 2)}};
  for (const auto& o : outs)
    for (const auto& i : ins)
      if (overlaps(o.p, o.n, i.p, i.n)) return LAPSUM_EINVAL;
  if (overlaps(outs[0].p, outs[0].n, outs[1].p, outs[1].n)) return LAPSUM_EINVAL;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  auto* offsets = reinterpret_cast<int32_t*>(ws + l.offsets);
  auto* rows = reinterpret_cast<int32_t*>(ws + l.rows);
  auto* slots = reinterpret_cast<int32_t*>(ws + l.slots);
  void* pre = keep && activation != LAPSUM_ACT_NONE ? ws + l.pre : nullptr;
  rc = lapsum_experts_plan(chosen, n, experts, offsets, rows, slots, ws + l.plan, l.x_rows - l.plan, stream);
  if (rc == LAPSUM_OK)
    rc = lapsum_experts_dispatch(x, dtype, tokens, k, dim, x_stride, slots, ws + l.x_rows, dim, stream);
  if (rc == LAPSUM_OK)
    rc = lapsum_experts_linear_fwd(ws + l.x_rows, dtype, n, dim, dim, w_in, experts, up, offsets, b_in, activation,
                                   nullptr, 0, ws + l.h, hidden, pre, up, status, stream);
  if (rc == LAPSUM_OK)
    rc = lapsum_experts_linear_fwd(ws + l.h, dtype, n, hidden, hidden, w_out, experts, dim_out, offsets, b_out,
                                   LAPSUM_ACT_NONE, nullptr, 0, ws + l.y, dim_out, nullptr, 0, status, stream);
  if (rc == LAPSUM_OK)
    rc = lapsum_experts_combine(ws + l.y, dtype, tokens, k, dim_out, dim_out, weights, rows, residual, residual_stride,
                                out, out_stride, stream);
  return rc;
}

// Scratch of the layer's backward: the rows' gradients and the products' own.  They
// are of the type: gy and gh are operands of the products, gx (which combine adds up
// in fp32) would be twice the bytes in fp32.
struct MlpBwdLayout {
  size_t gy, gh, gx, products, total;
};
static MlpBwdLayout mlp_bwd_layout(int64_t n, int experts, int64_t dim, int64_t up, int activation, int64_t dim_out) {
  MlpBwdLayout l;
  const int64_t hidden = activation == LAPSUM_ACT_SWIGLU ? up / 2 : up;
  l.gy = 0;
  l.gh = round256(2 * (size_t)n * dim_out);
  l.gx = l.gh + round256(2 * (size_t)n * hidden);
  l.products = l.gx + round256(2 * (size_t)n * dim);
  l.total = l.products + std::max(lapsum_experts_linear_bwd_workspace_size(n, experts, dim_out, LAPSUM_ACT_NONE, 1),
                                  lapsum_experts_linear_bwd_workspace_size(n, experts, up, activation, 1));
  return l;
}

size_t lapsum_experts_mlp_bwd_workspace_size(int64_t tokens, int k, int experts, int64_t dim, int64_t up, int activation,
                                             int64_t dim_out) {
  if (mlp_shape(LAPSUM_BF16, tokens, k, experts, dim, up, activation, dim_out) != LAPSUM_OK) return 0;
  return mlp_bwd_layout(tokens * k, experts, dim, up, activation, dim_out).total;
}

int lapsum_experts_mlp_bwd(const void* grad, int dtype, int64_t tokens, int64_t dim, int64_t grad_stride,
                           const float* weights, int k, const void* w_in, int experts, int64_t up, int activation,
                           const void* w_out, int64_t dim_out, const void* kept, int residual_is_x, void* grad_x,
                           float* grad_weights, void* grad_w_in, void* grad_b_in, void* grad_w_out, void* grad_b_out,
                           uint32_t* status, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = mlp_shape(dtype, tokens, k, experts, dim, up, activation, dim_out);
  if (rc != LAPSUM_OK) return rc;
  const int64_t n = tokens * k;
  const bool inner = grad_x || grad_w_in || grad_b_in, outer = inner || grad_w_out || grad_b_out;
  if (!grad || !weights || !w_in || !w_out || !kept || grad_stride < dim_out || (!outer && !grad_weights)) return LAPSUM_EINVAL;
  if (residual_is_x && dim != dim_out) return LAPSUM_EINVAL;
  if (!aligned(grad, 2) || !aligned(weights, 4) || !aligned(w_in, 16) || !aligned(w_out, 16) || !aligned(kept, 256) ||
      !aligned(grad_x, 16) || !aligned(grad_weights, 4) || !aligned(grad_w_in, 16) || !aligned(grad_b_in, 2) ||
      !aligned(grad_w_out, 16) || !aligned(grad_b_out, 2) || !aligned(status, 4))
    return LAPSUM_EINVAL;
  const MlpLayout l = mlp_layout(tokens, k, experts, dim, up, activation, dim_out, true);
  const MlpBwdLayout b = mlp_bwd_layout(n, experts, dim, up, activation, dim_out);
  const int64_t hidden = l.hidden;
  if (!workspace || workspace_bytes < b.total || !aligned(workspace, 256)) return LAPSUM_EWORKSPACE;
  const size_t wi = 2 * (size_t)experts * up * dim, wo = 2 * (size_t)experts * dim_out * hidden;
  struct {
    const void* p;
    size_t n;
  } outs[7] = {{grad_x, 2 * (size_t)tokens * dim}, {grad_weights, 4 * (size_t)n}, {grad_w_in, wi},
               {grad_b_in, 2 * (size_t)experts * up}, {grad_w_out, wo}, {grad_b_out, 2 * (size_t)experts * dim_out},
               {workspace, b.total}},
    ins[5] = {{grad, span(tokens, dim_out, grad_stride, 2)}, {weights, 4 * (size_t)n}, {w_in, wi}, {w_out, wo}, {kept, l.total}};
  for (int o = 0; o < 7; ++o) {
    for (const auto& i : ins)
      if (overlaps(outs[o].p, outs[o].n, i.p, i.n)) return LAPSUM_EINVAL;
    for (int q = 0; q < o; ++q)
      if (overlaps(outs[o].p, outs[o].n, outs[q].p, outs[q].n)) return LAPSUM_EINVAL;
  }
  const unsigned char* in = static_cast<const unsigned char*>(kept);
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  auto* offsets = reinterpret_cast<const int32_t*>(in + l.offsets);
  auto* rows = reinterpret_cast<const int32_t*>(in + l.rows);
  auto* slots = reinterpret_cast<const int32_t*>(in + l.slots);
  const void* pre = activation != LAPSUM_ACT_NONE ? in + l.pre : nullptr;
  const size_t left = workspace_bytes - b.products;
  rc = lapsum_experts_combine_bwd(grad, dtype, tokens, k, dim_out, grad_stride, in + l.y, dim_out, weights, rows, slots,
                                  outer ? ws + b.gy : nullptr, dim_out, grad_weights, stream);
  if (rc == LAPSUM_OK && outer)
    rc = lapsum_experts_linear_bwd(ws + b.gy, dtype, n, dim_out, dim_out, nullptr, in + l.h, hidden, hidden, w_out, experts,
                                   offsets, LAPSUM_ACT_NONE, inner ? ws + b.gh : nullptr, grad_w_out, grad_b_out, status,
                                   ws + b.products, left, stream);
  if (rc == LAPSUM_OK && inner)
    rc = lapsum_experts_linear_bwd(ws + b.gh, dtype, n, up, hidden, pre, in + l.x_rows, dim, dim, w_in, experts, offsets,
                                   activation, grad_x ? ws + b.gx : nullptr, grad_w_in, grad_b_in, status,
                                   ws + b.products, left, stream);
  if (rc == LAPSUM_OK && grad_x)
    rc = lapsum_experts_combine(ws + b.gx, dtype, tokens, k, dim, dim, nullptr, rows, residual_is_x ? grad : nullptr,
                                grad_stride, grad_x, dim, stream);
  return rc;
}

}  // extern "C"
