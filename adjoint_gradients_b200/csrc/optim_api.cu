// optim_api.cu -- the C ABI of the optimiser (declared in include/qml.h):
// argument checks, the table of work units and the order of launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>
#include <utility>
#include <vector>

#include "device_guard.h"
#include "optim.cuh"
#include "qml.h"

using namespace qml;

namespace {

constexpr size_t kOptAlign = 256;
constexpr int kNormPerSm = 4;  // blocks of the norm's launches, per SM: as many as are resident at its 64 registers

// Rounds of a unit of work.  A block pays for its start once a unit (its
// record, the step's factors, the random key, the unit's scales: some 2 us of
// dependent loads), so units are as long as leaves one for every block that is
// resident at once (3 an SM), or a whole number of them, up to a cap.  128M fp32
// elements with 1 / 2 / 4 / 8 / 16 rounds (the 8-bit kernel as it was then): 8-bit
// 746 / 494 / 419 / 389 / 385 us; full states, whose start is shorter, 611 / 537 /
// 526 / 538 / 544.  fp64 has one block an SM, its units are cut for three all the
// same: no other number has been measured (4M elements 47 us, floor 34).
constexpr long long kResident = 148 * 3;
int rounds_for(long long total, bool bits8) {
  const long long rounds = (total + kOptChunk - 1) / kOptChunk, cap = bits8 ? kOptMaxRounds : 4;
  const long long waves = std::max(1ll, (rounds + kResident * cap - 1) / (kResident * cap));
  return (int)std::max(1ll, (rounds + kResident * waves - 1) / (kResident * waves));
}

// Blocks of 256 elements up to which a step is one launch of one cluster.
// Device time a step, one launch against the general kernels (clipped: two
// launches), full / 8-bit states: 60,000 fp32 elements 3.2 / 3.9 against 3.8 /
// 4.7 us, clipped 4.1 / 4.9 against 7.8 / 8.5; 6,000 clipped 3.3 against 8.1.
// fp64 at 60,000 loses a little where the step is not clipped, 5.9 against 5.5:
// the units are cut when the handle is made, before it is known whether it will be.
constexpr long long kSmallBlocks = kOptSmallCluster * kOptSmallWarps;

constexpr long long kMaxElements = 1ll << 36;  // of a handle: what 180 GB of states cannot hold

size_t round_up(size_t v) { return (v + kOptAlign - 1) / kOptAlign * kOptAlign; }

size_t type_size(int t) { return t == QML_F64 ? 8 : t == QML_F32 ? 4 : 2; }

bool off(const void* p, size_t a) { return ((uintptr_t)p) % a != 0; }

// Whether a factor is finite in the type that the step computes in.
bool finite_in(bool f64, double x) { return std::isfinite(f64 ? x : (double)(float)x); }

bool negative_or_not_finite(bool f64, double x) { return !(x >= 0.0) || !finite_in(f64, x); }

// Tensors of one launch: one combination of types, at most as many as the
// kernel parameters hold gradient pointers.
struct Launch {
  OptCombo combo;
  int chunk0, n_chunks, slot0, n_slots;
};

}  // namespace

struct qml_opt {
  qml_opt_config cfg{};
  int device = 0;
  bool f64 = false;
  bool small = false;  // steps run in one launch
  int cluster = 8;     // of at most so many thread blocks
  int sms = 0;
  std::vector<int> order;  // slot (launch order) -> tensor
  std::vector<int> grad_type;  // by tensor
  std::vector<long long> numel;
  std::vector<OptChunk> chunks;
  std::vector<Launch> launches;
  std::vector<const void*> grads;  // scratch: the pointers in launch order
  char* ws = nullptr;
  long long launched = 0;

  size_t chunk_off() const { return round_up(sizeof(OptCtrl)); }
  size_t part_off() const { return chunk_off() + round_up(sizeof(OptChunk) * chunks.size()); }
  size_t bytes() const { return part_off() + round_up(sizeof(double) * (size_t)norm_grid() * launches.size()); }
  int norm_grid() const { return kNormPerSm * sms; }
  OptCtrl* ctrl() const { return reinterpret_cast<OptCtrl*>(ws); }
  const OptChunk* table() const { return reinterpret_cast<const OptChunk*>(ws + chunk_off()); }
};

namespace {

// Checks one tensor; the pointer ranges of its buffers go to `used`.
qml_status check_tensor(const qml_opt_tensor& t, bool bits8, std::vector<std::pair<uintptr_t, uintptr_t>>* used) {
  if (t.dtype < QML_F32 || t.dtype > QML_F16 || t.grad_dtype < QML_F32 || t.grad_dtype > QML_F16)
    return QML_ERR_INVALID_ARG;
  const bool half = t.dtype == QML_BF16 || t.dtype == QML_F16;
  if (t.grad_dtype != t.dtype && !(half && t.grad_dtype == QML_F32)) return QML_ERR_UNSUPPORTED;
  if (t.dtype == QML_F64 && bits8) return QML_ERR_UNSUPPORTED;
  if (t.master && !half) return QML_ERR_UNSUPPORTED;
  const bool f64 = t.dtype == QML_F64;
  if (negative_or_not_finite(f64, t.lr_scale) || negative_or_not_finite(f64, t.weight_decay)) return QML_ERR_INVALID_ARG;
  if (t.numel < 0 || t.numel > kMaxElements) return QML_ERR_INVALID_ARG;
  if (t.numel == 0) return QML_OK;
  const size_t n = (size_t)t.numel, ps = type_size(t.dtype);
  const size_t ss = bits8 ? 1 : t.dtype == QML_F64 ? 8 : 4, blocks = (n + kOptBlock - 1) / kOptBlock;
  if (!t.param || !t.m || !t.v || off(t.param, ps) || off(t.master, 4) || off(t.m, ss) || off(t.v, ss))
    return QML_ERR_INVALID_ARG;
  if (bits8 && (!t.m_scale || !t.v_scale || off(t.m_scale, 4) || off(t.v_scale, 4))) return QML_ERR_INVALID_ARG;
  auto add = [&](const void* p, size_t bytes) {
    if (p) used->push_back({(uintptr_t)p, (uintptr_t)p + bytes});
  };
  add(t.param, n * ps);
  add(t.master, n * 4);
  add(t.m, n * ss);
  add(t.v, n * ss);
  if (bits8) add(t.m_scale, blocks * 4), add(t.v_scale, blocks * 4);
  return QML_OK;
}

OptCombo combo_of(const qml_opt_tensor& t, bool bits8) {
  return OptCombo{t.dtype, t.grad_dtype, t.master ? 1 : 0, bits8 ? 1 : 0};
}

int combo_key(const OptCombo& c) { return c.param * 64 + c.grad * 8 + c.master; }

qml_status build(qml_opt* o, int n_tensors, const qml_opt_tensor* ts) {
  const bool bits8 = o->cfg.state == QML_STATE_8BIT;
  std::vector<std::pair<uintptr_t, uintptr_t>> used;
  int n64 = 0;
  long long total = 0, n_chunks = 0;
  for (int i = 0; i < n_tensors; ++i) {
    const qml_status st = check_tensor(ts[i], bits8, &used);
    if (st != QML_OK) return st;
    n64 += ts[i].dtype == QML_F64;
    total += ts[i].numel;
    if (total > kMaxElements) return QML_ERR_INVALID_ARG;
  }
  long long blocks = 0;
  bool one_combo = true;
  for (int i = 0; i < n_tensors; ++i) {
    blocks += (ts[i].numel + kOptBlock - 1) / kOptBlock;
    one_combo = one_combo && combo_key(combo_of(ts[i], bits8)) == combo_key(combo_of(ts[0], bits8));
  }
  o->small = blocks <= kSmallBlocks && one_combo && n_tensors <= kOptCaps[0];
  const int unit = o->small ? kOptBlock : kOptChunk * rounds_for(total, bits8);
  for (int i = 0; i < n_tensors; ++i) n_chunks += (ts[i].numel + unit - 1) / unit;
  if (n64 && n64 < n_tensors) return QML_ERR_UNSUPPORTED;
  std::sort(used.begin(), used.end());
  for (size_t i = 1; i < used.size(); ++i)
    if (used[i].first < used[i - 1].second) return QML_ERR_INVALID_ARG;  // two buffers overlap
  o->f64 = n64 > 0;
  o->order.resize((size_t)n_tensors);
  for (int i = 0; i < n_tensors; ++i) o->order[(size_t)i] = i;
  std::stable_sort(o->order.begin(), o->order.end(), [&](int a, int b) {
    return combo_key(combo_of(ts[a], bits8)) < combo_key(combo_of(ts[b], bits8));
  });
  o->chunks.reserve((size_t)n_chunks);
  o->numel.resize((size_t)n_tensors);
  o->grad_type.resize((size_t)n_tensors);
  o->grads.resize((size_t)n_tensors);
  for (int slot = 0; slot < n_tensors; ++slot) {
    const int i = o->order[(size_t)slot];
    const qml_opt_tensor& t = ts[i];
    o->numel[(size_t)i] = t.numel;
    o->grad_type[(size_t)i] = t.grad_dtype;
    const OptCombo c = combo_of(t, bits8);
    if (o->launches.empty() || combo_key(o->launches.back().combo) != combo_key(c) ||
        o->launches.back().n_slots == kOptCaps[1])
      o->launches.push_back({c, (int)o->chunks.size(), 0, slot, 0});
    Launch& l = o->launches.back();
    ++l.n_slots;
    const size_t ps = type_size(t.dtype), ss = bits8 ? 1 : t.dtype == QML_F64 ? 8 : 4;
    const size_t pa = std::min<size_t>(8 * ps, 32), sa = bits8 ? 16 : 32;
    const bool aligned = !off(t.param, pa) && !off(t.master, 32) && !off(t.m, sa) && !off(t.v, sa);
    for (long long at = 0; at < t.numel; at += unit) {
      OptChunk k{};
      k.p = static_cast<char*>(t.param) + (size_t)at * ps;
      k.master = t.master ? static_cast<float*>(t.master) + at : nullptr;
      k.m = static_cast<char*>(t.m) + (size_t)at * ss;
      k.v = static_cast<char*>(t.v) + (size_t)at * ss;
      k.m_scale = bits8 ? t.m_scale + at / kOptBlock : nullptr;
      k.v_scale = bits8 ? t.v_scale + at / kOptBlock : nullptr;
      k.first = at;
      k.count = (int)std::min<long long>(unit, t.numel - at);
      k.slot = slot;
      k.tensor = (uint32_t)i;
      k.aligned = aligned ? 1 : 0;
      k.lr_scale = t.lr_scale;
      k.decay = t.weight_decay;
      k.lr_scale_f = (float)t.lr_scale;
      k.decay_f = (float)t.weight_decay;
      o->chunks.push_back(k);
      ++l.n_chunks;
    }
  }
  return QML_OK;
}

// The gradients in launch order, checked.
qml_status take_grads(qml_opt* o, const void* const* grads) {
  for (size_t slot = 0; slot < o->order.size(); ++slot) {
    const size_t i = (size_t)o->order[slot];
    if (off(grads[i], type_size(o->grad_type[i]))) return QML_ERR_INVALID_ARG;
    o->grads[slot] = grads[i];
  }
  return QML_OK;
}

qml_status run_norm(qml_opt* o, double grad_scale, double max_norm, void* norm, bool set_clip, cudaStream_t s) {
  OptNormArgs a{};
  a.ctrl = o->ctrl();
  a.grad_scale = grad_scale;
  a.max_norm = max_norm;
  a.partials = reinterpret_cast<double*>(o->ws + o->part_off());
  a.norm = norm;
  a.norm64 = o->f64 ? 1 : 0;
  a.set_clip = set_clip ? 1 : 0;
  for (const Launch& l : o->launches) a.n_part += std::max(1, std::min(l.n_chunks, o->norm_grid()));
  for (size_t i = 0; i < o->launches.size(); ++i) {
    const Launch& l = o->launches[i];
    const int grid = std::max(1, std::min(l.n_chunks, o->norm_grid()));
    a.chunks = o->table() + l.chunk0;
    a.n_chunks = l.n_chunks;
    a.slot0 = l.slot0;
    a.grad_type = l.combo.grad;
    a.last = i + 1 == o->launches.size();
    if (launch_opt_norm(a, o->grads.data() + l.slot0, l.n_slots, grid, s) != cudaSuccess) return QML_ERR_CUDA;
    ++o->launched;
    a.part0 += grid;
  }
  return QML_OK;
}

qml_status ready(qml_opt* o, const void* const* grads, double grad_scale) {
  if (!o || !grads || !std::isfinite(grad_scale)) return QML_ERR_INVALID_ARG;
  if (!o->ws) return QML_ERR_WORKSPACE;
  return QML_OK;
}

}  // namespace

extern "C" {

qml_status qml_opt_create(const qml_opt_config* cfg, int n_tensors, const qml_opt_tensor* tensors, int device,
                          qml_opt** out) {
  if (!out) return QML_ERR_INVALID_ARG;
  *out = nullptr;
  if (!cfg || !tensors || n_tensors < 1 || n_tensors > QML_MAX_OPT_TENSORS || device < 0) return QML_ERR_INVALID_ARG;
  if (cfg->state != QML_STATE_FULL && cfg->state != QML_STATE_8BIT) return QML_ERR_INVALID_ARG;
  if (!(cfg->beta1 >= 0.0 && cfg->beta1 < 1.0) || !(cfg->beta2 >= 0.0 && cfg->beta2 < 1.0)) return QML_ERR_INVALID_ARG;
  if (!(cfg->eps >= 1e-30 && cfg->eps <= 1e30)) return QML_ERR_INVALID_ARG;  // (the quotient's range in fp32)
  qml_opt* o = nullptr;
  try {  // the tables are host vectors: running out of host memory is an error code, too
    o = new qml_opt();
    o->cfg = *cfg;
    o->device = device;
    const qml_status st = build(o, n_tensors, tensors);
    if (st != QML_OK) {
      delete o;
      return st;
    }
  } catch (const std::bad_alloc&) {
    delete o;
    return QML_ERR_INVALID_ARG;
  }
  int sms = 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) {
    cudaGetLastError();  // no such device here: qml_opt_set_workspace says so
    sms = 148;
  }
  o->sms = sms;
  *out = o;
  return QML_OK;
}

qml_status qml_opt_destroy(qml_opt* o) {
  if (!o) return QML_ERR_INVALID_ARG;
  delete o;
  return QML_OK;
}

size_t qml_opt_workspace_bytes(const qml_opt* o) { return o ? o->bytes() : 0; }

qml_status qml_opt_set_workspace(qml_opt* o, void* ws, size_t bytes, void* stream) {
  if (!o || !ws || off(ws, kOptAlign)) return QML_ERR_INVALID_ARG;
  if (bytes < o->bytes()) return QML_ERR_WORKSPACE;
  DeviceGuard g(o->device);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int now = -1;
  if (cudaGetDevice(&now) != cudaSuccess || now != o->device) {  // the handle's device is not there
    cudaGetLastError();
    return QML_ERR_CUDA;
  }
  o->ws = static_cast<char*>(ws);
  if (o->small) {
    o->cluster = opt_cluster_limit(o->launches[0].combo);
    o->small = (long long)o->chunks.size() <= (long long)o->cluster * kOptSmallWarps;
  }
  cudaError_t e = cudaMemsetAsync(o->ws, 0, sizeof(OptCtrl), s);
  if (e == cudaSuccess && !o->chunks.empty())
    e = cudaMemcpyAsync(o->ws + o->chunk_off(), o->chunks.data(), sizeof(OptChunk) * o->chunks.size(),
                        cudaMemcpyHostToDevice, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess || qml_opt_set_step(o, 0, stream) != QML_OK) {
    cudaGetLastError();
    o->ws = nullptr;
    return QML_ERR_CUDA;
  }
  return QML_OK;
}

qml_status qml_opt_set_step(qml_opt* o, long long t, void* stream) {
  if (!o || t < 0) return QML_ERR_INVALID_ARG;
  if (!o->ws) return QML_ERR_WORKSPACE;
  DeviceGuard g(o->device);
  ++o->launched;
  return launch_opt_set(o->ctrl(), t, o->cfg.beta1, o->cfg.beta2, o->cfg.seed,
                        static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? QML_OK
             : QML_ERR_CUDA;
}

qml_status qml_opt_get_step(qml_opt* o, long long* t, void* stream) {
  if (!o || !t) return QML_ERR_INVALID_ARG;
  if (!o->ws) return QML_ERR_WORKSPACE;
  DeviceGuard g(o->device);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemcpyAsync(t, &o->ctrl()->t, sizeof(*t), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  return e == cudaSuccess ? QML_OK : QML_ERR_CUDA;
}

qml_status qml_opt_step(qml_opt* o, const void* const* grads, double lr, const void* lr_dev, double grad_scale,
                        double max_norm, void* norm_dev, void* stream) {
  qml_status st = ready(o, grads, grad_scale);
  if (st != QML_OK) return st;
  if (!finite_in(o->f64, grad_scale) || (!lr_dev && negative_or_not_finite(o->f64, lr))) return QML_ERR_INVALID_ARG;
  const size_t real = o->f64 ? 8 : 4;
  if (off(lr_dev, real) || off(norm_dev, real)) return QML_ERR_INVALID_ARG;
  if (!(max_norm >= 0.0) || (norm_dev && max_norm == 0.0)) return QML_ERR_INVALID_ARG;
  st = take_grads(o, grads);
  if (st != QML_OK) return st;
  DeviceGuard g(o->device);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool clipped = max_norm > 0.0;
  if (clipped && !o->small) {
    st = run_norm(o, grad_scale, max_norm, norm_dev, true, s);
    if (st != QML_OK) return st;
  }
  OptSettings a{};
  a.ctrl = o->ctrl();
  a.lr = lr;
  a.lr_dev = lr_dev;
  a.beta1 = o->cfg.beta1;
  a.beta2 = o->cfg.beta2;
  a.eps = o->cfg.eps;
  a.grad_scale = grad_scale;
  a.seed = o->cfg.seed;
  a.clipped = clipped ? 1 : 0;
  for (size_t i = 0; i < o->launches.size(); ++i) {
    const Launch& l = o->launches[i];
    a.chunks = o->table() + l.chunk0;
    a.n_chunks = l.n_chunks;
    a.slot0 = l.slot0;
    a.last = i + 1 == o->launches.size();
    const OptClipArgs clip{grad_scale, max_norm, norm_dev, o->f64 ? 1 : 0, o->cluster};
    if (launch_opt_step(l.combo, a, o->small ? &clip : nullptr, o->grads.data() + l.slot0, l.n_slots, s) !=
        cudaSuccess)
      return QML_ERR_CUDA;
    ++o->launched;
  }
  return QML_OK;
}

qml_status qml_opt_grad_norm(qml_opt* o, const void* const* grads, double grad_scale, void* norm_dev, void* stream) {
  qml_status st = ready(o, grads, grad_scale);
  if (st != QML_OK) return st;
  if (!norm_dev || off(norm_dev, o->f64 ? 8 : 4)) return QML_ERR_INVALID_ARG;
  st = take_grads(o, grads);
  if (st != QML_OK) return st;
  DeviceGuard g(o->device);
  return run_norm(o, grad_scale, 0.0, norm_dev, false, static_cast<cudaStream_t>(stream));
}

qml_status qml_opt_sync(qml_opt* o, void* stream) {
  if (!o) return QML_ERR_INVALID_ARG;
  if (!o->ws) return QML_ERR_WORKSPACE;
  DeviceGuard g(o->device);
  // all on `stream`: on the default stream the clearing could come after a later
  // call's error, and wait for work that is none of this handle's
  unsigned word = 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemcpyAsync(&word, &o->ctrl()->status, sizeof(word), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess && word) e = cudaMemsetAsync(&o->ctrl()->status, 0, sizeof(word), s);
  if (e != cudaSuccess) return QML_ERR_CUDA;
  for (int code = 1; code < 32; ++code)
    if (word & (1u << code)) return static_cast<qml_status>(code);
  return QML_OK;
}

long long qml_opt_launch_count(const qml_opt* o) { return o ? o->launched : -1; }

}  // extern "C"
