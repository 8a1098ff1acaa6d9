// api.cu -- the C ABI of libqml (declared in include/qml.h).
//
// Host-side only: argument checks, the pass schedule, the workspace layout,
// and the order of kernel launches.  Every arithmetic step of the forward and
// backward paths runs in the kernels of kernels.cu.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstdlib>
#include <cstring>
#include <new>
#include <string>
#include <vector>

#include "device_guard.h"
#include "kernels.cuh"
#include "plan.hpp"
#include "qml.h"

using namespace qml;

namespace {

constexpr size_t kAlign = 256;
size_t align_up(size_t v) { return (v + kAlign - 1) & ~(kAlign - 1); }

struct Layout {
  size_t status, passes, slot_pass, slot_index;
  size_t coef_fwd, coef_inv, enc, dummy, exp_partial, partials, obs_groups, obs_terms, ckpt;
  size_t ckpt_exps;  // QML_STORE_INT8 slots: exponent bytes
  size_t scratch, dummy2, sub_passes, sub_slot_pass, sub_slot_index;  // CNOT entanglers only
  size_t passes_split, undo, s_rot, s_lay, s_gfix, s_dqf, s_dqb, rscale;  // split form (fp32 only)
  size_t fault_theta;  // QML_FAULT=nan_theta, fp64: a copy of theta with a NaN angle
  size_t s_dq64f, s_dq64b, rscale64;  // split form, fp64 contexts
  size_t base_total;
  // host-step extras
  size_t h_psi, h_lam, h_x, h_theta, h_y, h_E, h_g, h_loss, h_grad;
  size_t host_total;
};

}  // namespace

struct qml_ctx {
  qml_config cfg{};
  int device = 0;
  Plan plan;
  std::vector<DevPass> dpass;
  // the same passes in split form (OP_RY / OP_DIAG), used by fp32 contexts
  // without re-uploading or CNOT entanglers
  std::vector<DevPass> dpass_split;
  std::vector<int> undo;  // split form: [L][n] backward un-apply order of each layer's qubits
  size_t smem = 0;
  size_t smem_multi = 0;  // one-launch split passes of single-tile circuits
  bool probed = false, dev_ok = false;
  bool slow = false;  // the plan puts a batch-unit bit in registers (n < 5)
  int region = 0;     // constant-memory coefficient region
  int sms = 148, grid_fwd = 0, grid_bwd = 0;
  char* ws = nullptr;
  size_t ws_bytes = 0;
  Layout lay{};
  std::vector<int> ckpt_batch;  // batch last written to each slot, -1 = never
  long long N = 0;
  long long launches = 0;
  bool timing = false;
  struct Span {
    cudaEvent_t a, b;
    bool bwd;
    int passes;
  };
  std::vector<Span> spans;
  std::vector<cudaEvent_t> spare;
  // tensor maps of the passes that load by tensor copies, keyed by the view
  // of the tile and by the buffers they were encoded for
  struct MapEntry {
    DevPass view;  // a pass with this view
    bool backward;
    int B;
    const void *buf0, *buf1;
    PassMaps maps;
  };
  std::vector<MapEntry> maps;
  // observable (empty: Z0); uploaded to the workspace before its next use
  std::vector<ObsGroup> obs_groups;
  std::vector<ObsTerm> obs_terms;
  bool obs_dirty = false;
  // entangler of every layer (CZ bonds); chain = the default (q, q+1) ladder
  Bonds bonds;
  uint32_t nb[kMaxQubits] = {0}, nbhi[kMaxQubits] = {0};
  bool reupload = false;  // every layer starts with the encoding again
  // CNOT entanglers (qml_set_entangler_cnot): every layer's rotations run as
  // the passes of a one-layer schedule (sub[v], v = 2 * encodes + stores the
  // standard layout), and the layer's CNOT list as a gather between buffers
  bool cnot = false;
  std::vector<std::pair<int, int>> cnot_pairs;
  LinMap cnot_fwd{}, cnot_bwd{};  // M^-1 (apply) and M (un-apply) of a layer's CNOT list, on addresses
  LinMap cnot_fwd_q{}, cnot_bwd_q{};  // the same on qubit bits (fp64 mode: standard order)
  std::vector<uint32_t> sub_mask;     // fp64 tiles of the one-layer passes
  Plan plan1;
  std::vector<DevPass> sub[4];
  bool sub_uploaded = false;
  // Fused CNOT layers (fp32, two qubit sets, a list whose map factors as
  // M2 M1, see plan.hpp): plan and dpass are then the fused schedule, whose
  // passes apply M1 and M2 inside their tiles; re-uploading still takes the
  // one-layer schedules above.
  bool cnot_fused = false;
  CnotLayers cnot_map{};  // M1, M2 of the fused schedule
  // qml_step_host replays a CUDA graph of its copies and launches once the
  // same call (buffers, batch, settings) has run eagerly; gen counts changes
  // of the settings a captured step depends on
  struct HostGraph {
    cudaGraphExec_t exec = nullptr;
    const void* key[7] = {};
    int B = 0;
    unsigned gen = 0;
    long long launches = 0;  // kernel launches inside the graph
    bool seen = false;       // the keyed call ran eagerly once
    bool failed = false;     // its capture failed: stay eager
  } hg;
  unsigned gen = 1;
  cudaStream_t cap = nullptr;  // capture stream of the host-step graph
  // the theta buffer (and settings generation) the fp32 coefficient tables
  // were last prepared from by a forward call; the backward of the same
  // buffer reuses them
  const void* prep_theta = nullptr;
  unsigned prep_gen = 0;
  bool f64 = false;       // fp64 compute mode (qml_create_f64)
  // host-side fault injection for tests of the error paths (QML_FAULT at create)
  enum Fault { FAULT_NONE, FAULT_ALLOC, FAULT_CKPT, FAULT_NAN } fault = FAULT_NONE;
  std::vector<uint32_t> f64_mask;  // fp64: tile qubits of each pass
  int f64_tmax = 0;                // fp64: largest tile (qubits)
};

namespace {

// Probe the device once: shared-memory opt-in, occupancy, persistent grid size.
void ensure_device(qml_ctx* c) {
  if (c->probed) return;
  c->probed = true;
  if (c->f64) {
    int bf = 0, bb = 0, sms = 0;
    DeviceGuard g(c->device);
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, c->device) != cudaSuccess ||
        pass64_setup(c->f64_tmax, &bf, &bb) != cudaSuccess ||
        bf < 1 || bb < 1) {
      cudaGetLastError();
      c->dev_ok = false;
      c->grid_fwd = c->grid_bwd = c->sms;
      return;
    }
    c->sms = sms;
    c->grid_fwd = c->sms * bf;
    c->grid_bwd = c->sms * bb;
    c->dev_ok = true;
    return;
  }
  // every pass of a context loads the same way: tensor copies for n > 12
  const bool tma = !c->dpass.empty() && c->dpass[0].tma;
  const int mode = tma ? 2 : c->slow ? 0 : 1;
  // the function attribute is shared by all contexts: set it for the largest pass
  const size_t smem_thr = pass_smem_bytes(kMaxSlots, false), smem_tma = pass_smem_bytes(kMaxSlots, true);
  c->smem_multi = pass_multi_smem_bytes();
  c->smem = tma ? smem_tma : smem_thr;
  int sms = 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, c->device) != cudaSuccess) {
    cudaGetLastError();
    c->dev_ok = false;
    c->grid_fwd = c->sms * 3;
    c->grid_bwd = c->sms * 2;
    return;
  }
  DeviceGuard g(c->device);
  c->sms = sms;
  int of = 0, ob = 0;
  if (set_pass_smem_attr(std::max(smem_thr, c->smem_multi), smem_tma) != cudaSuccess || pass_occupancy(false, mode, c->smem, &of) != cudaSuccess ||
      pass_occupancy(true, mode, c->smem, &ob) != cudaSuccess || of < 1 || ob < 1) {
    cudaGetLastError();
    c->dev_ok = false;
    c->grid_fwd = c->sms * 3;
    c->grid_bwd = c->sms * 2;
    return;
  }
  c->grid_fwd = c->sms * of;
  c->grid_bwd = c->sms * ob;
  c->dev_ok = true;
}

// Bytes per amplitude of a checkpoint slot.
size_t slot_bytes(const qml_ctx* c) {
  if (c->cfg.storage == QML_STORE_INT8) return 2;  // and an exponent byte a block, kept apart
  return c->cfg.storage == QML_STORE_FP64 ? 16 : c->cfg.storage == QML_STORE_BF16 ? 4 : 8;
}

void compute_layout(qml_ctx* c) {
  const int n = c->cfg.n_qubits, L = c->cfg.n_layers, Bm = c->cfg.max_batch;
  const long long N = 1ll << n;
  const size_t U = (size_t)(Bm + 1) / 2;
  Layout& l = c->lay;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    size_t at = o;
    o = align_up(o + bytes);
    return at;
  };
  l.status = take(64);
  l.passes = take(sizeof(DevPass) * c->dpass.size());
  l.slot_pass = take(sizeof(int) * (size_t)L * n);
  l.slot_index = take(sizeof(int) * (size_t)L * n);
  l.coef_fwd = take(sizeof(CoefRegion) * std::max(c->dpass.size(), c->sub[0].size()));
  l.coef_inv = take(sizeof(CoefRegion) * std::max(c->dpass.size(), c->sub[0].size()));
  l.enc = take(sizeof(float2) * 2 * U * n);
  l.dummy = take(sizeof(float2) * (size_t)N);
  // (fp32: also room for one partial per 4096-position tile and sample, the Z0 epilogue's)
  l.exp_partial = take(sizeof(double) * (c->f64 ? expect64_partial_count(Bm, n)
                                                : std::max(expect_partial_count(Bm, n),
                                                           (size_t)Bm << (n > kTileBits ? n - kTileBits : 0))));
  size_t nparts = 0;
  for (const DevPass& p : c->dpass) nparts += (size_t)c->grid_bwd * p.nslots * 3;
  l.partials = take((c->f64 ? sizeof(double) : sizeof(float)) * std::max<size_t>(1, nparts));
  l.obs_groups = take(sizeof(ObsGroup) * QML_MAX_OBS_TERMS);
  l.obs_terms = take(sizeof(ObsTerm) * QML_MAX_OBS_TERMS);
  const size_t slot_elem = slot_bytes(c);
  l.ckpt = take(slot_elem * (size_t)c->plan.n_ckpt * Bm * (size_t)N + 16);
  l.ckpt_exps = c->cfg.storage == QML_STORE_INT8 ? take(slot8_blocks(n) * (size_t)c->plan.n_ckpt * Bm + 16) : 0;
  if (c->cnot) {  // second state buffer and partner plane for the gathers, the one-layer schedules
    l.scratch = take((c->f64 ? sizeof(double2) : sizeof(float2)) * (size_t)Bm * N);
    l.dummy2 = take(sizeof(float2) * (size_t)N);
    l.sub_passes = take(sizeof(DevPass) * 4 * c->sub[0].size());
    l.sub_slot_pass = take(sizeof(int) * (size_t)n);
    l.sub_slot_index = take(sizeof(int) * (size_t)n);
  }
  l.passes_split = take(sizeof(DevPass) * c->dpass_split.size());
  l.undo = take(sizeof(int) * (size_t)L * n);
  l.s_rot = take(sizeof(SplitRot) * (size_t)L * n);
  l.s_lay = take(sizeof(SplitLayer) * 2 * (size_t)L);  // per layer, or per layer and set (fused CNOT)
  l.s_gfix = take(sizeof(double) * 2 * (size_t)L * n);
  if (!c->f64) {
    // per diagonal op: L + 1 of them, or 4 L in the fused CNOT schedule
    l.s_dqf = take(sizeof(float2) * 2 * (size_t)(4 * L + 1) * n);
    l.s_dqb = take(sizeof(float2) * 2 * (size_t)(4 * L + 1) * n);
    l.rscale = take(sizeof(float) * c->dpass_split.size());
  } else {
    l.s_dq64f = take(sizeof(double2) * 2 * (size_t)(L + 1) * n);
    l.s_dq64b = take(sizeof(double2) * 2 * (size_t)(L + 1) * n);
    l.rscale64 = take(sizeof(double) * c->dpass_split.size());
  }
  if (c->f64 && c->fault == qml_ctx::FAULT_NAN) l.fault_theta = take(sizeof(double) * 3 * (size_t)L * n);
  l.base_total = o;
  const size_t fe = c->f64 ? sizeof(double) : sizeof(float);  // real element of the host-step buffers
  l.h_psi = take(2 * fe * (size_t)Bm * N);
  l.h_lam = take(2 * fe * (size_t)Bm * N);
  l.h_x = take(fe * (size_t)Bm * n);
  l.h_theta = take(fe * (size_t)L * n * 3);
  l.h_y = take(fe * (size_t)Bm);
  l.h_E = take(fe * (size_t)Bm);
  l.h_g = take(fe * (size_t)Bm);
  l.h_loss = take(fe * 4);
  l.h_grad = take(fe * (size_t)L * n * 3);
  l.host_total = o;
  // gradient partial offsets per pass
  long long off = 0;
  for (size_t i = 0; i < c->dpass.size(); ++i) {
    c->dpass[i].partial_off = off;
    if (i < c->dpass_split.size()) c->dpass_split[i].partial_off = off;
    off += (long long)c->grid_bwd * c->dpass[i].nslots * 3;
  }
  // one-layer schedules: one layer's partials at a time, in the same area
  for (auto& v : c->sub) {
    long long o2 = 0;
    for (DevPass& p : v) {
      p.partial_off = o2;
      o2 += (long long)c->grid_bwd * p.nslots * 3;
    }
  }
  c->sub_uploaded = false;
}

cudaEvent_t take_event(qml_ctx* c) {
  if (!c->spare.empty()) {
    cudaEvent_t e = c->spare.back();
    c->spare.pop_back();
    return e;
  }
  cudaEvent_t e = nullptr;
  if (cudaEventCreate(&e) != cudaSuccess) return nullptr;
  return e;
}

// A timing event on s; inside a stream capture it becomes an event-record
// node of the graph (so every replay records it).  A failed record is
// cleared, so that it is not reported by the next launch check.
bool record_span_event(cudaEvent_t ev, cudaStream_t s) {
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(s, &cs) != cudaSuccess) cs = cudaStreamCaptureStatusNone;
  const cudaError_t e = cs == cudaStreamCaptureStatusActive ? cudaEventRecordWithFlags(ev, s, cudaEventRecordExternal)
                                                            : cudaEventRecord(ev, s);
  if (e != cudaSuccess) cudaGetLastError();
  return e == cudaSuccess;
}

// Record the start of a run of pass launches; returns false if timing is off.
bool span_begin(qml_ctx* c, cudaStream_t s, qml_ctx::Span* sp, bool bwd) {
  if (!c->timing) return false;
  sp->a = take_event(c);
  sp->b = take_event(c);
  sp->bwd = bwd;
  sp->passes = (int)c->dpass.size();
  if (!sp->a || !sp->b) return false;
  return record_span_event(sp->a, s);
}

void span_end(qml_ctx* c, cudaStream_t s, qml_ctx::Span* sp) {
  if (record_span_event(sp->b, s)) c->spans.push_back(*sp);
}

bool misaligned(const void* p, size_t a) { return ((uintptr_t)p) % a != 0; }

qml_status cuda_status(cudaError_t e) { return e == cudaSuccess ? QML_OK : QML_ERR_CUDA; }

template <class T>
T* at(qml_ctx* c, size_t off) {
  return reinterpret_cast<T*>(c->ws + off);
}

// 8-bit checkpoint slots are written and restored between pass launches.
bool int8_slots(const qml_ctx* c) { return c->cfg.storage == QML_STORE_INT8; }
int8_t* slot8_codes(qml_ctx* c, int m) {
  return reinterpret_cast<int8_t*>(c->ws + c->lay.ckpt) + 2 * (size_t)m * c->cfg.max_batch * (size_t)c->N;
}
uint8_t* slot8_exps(qml_ctx* c, int m) {
  return reinterpret_cast<uint8_t*>(c->ws + c->lay.ckpt_exps) +
         (size_t)m * c->cfg.max_batch * slot8_blocks(c->cfg.n_qubits);
}

// fp32 contexts run the split form unless a mode needs the fused SU(2)
// (re-uploading folds per-sample encodings into the rotations; CNOT layers
// run as one-layer schedules; 8-bit slots need a launch per pass, which the
// split form of single-tile circuits does not have).
bool use_split(const qml_ctx* c) {
  return !c->f64 && !c->reupload && (!c->cnot || c->cnot_fused) &&
         !(int8_slots(c) && c->plan.n_ckpt > 0 && c->cfg.n_qubits <= kTileBits);
}
// CNOT entanglers through the fused schedule (the generic pass loop), or the
// one-layer schedules with a gather per layer
bool cnot_fused_now(const qml_ctx* c) { return c->cnot && c->cnot_fused && !c->reupload; }
// fp64 contexts: the same rule
bool use_split64(const qml_ctx* c) { return c->f64 && !c->reupload && !c->cnot; }

const std::vector<DevPass>& fp32_passes(const qml_ctx* c) { return use_split(c) ? c->dpass_split : c->dpass; }
// The Z0 expectation fused into the last forward pass: split-form fp32
// passes with the Z0 observable over the standard order (at most two qubit
// sets: no working-state permutation), CZ entanglers.
bool fused_z0(const qml_ctx* c) { return use_split(c) && !c->cnot && c->obs_terms.empty() && c->plan.n_sets <= 2; }

// Readiness of a context for a call with batch B; f64 is the precision the
// call is made for (a context computes in one precision only).
qml_status check_ready(qml_ctx* c, int B, bool f64 = false) {
  if (!c) return QML_ERR_INVALID_ARG;
  if (c->f64 != f64) return QML_ERR_UNSUPPORTED;
  if (B < 1 || B > c->cfg.max_batch) return QML_ERR_INVALID_ARG;
  if (!c->ws) return QML_ERR_WORKSPACE;
  if (!c->dev_ok) return QML_ERR_CUDA;
  return QML_OK;
}

bool same_tma_view(const DevPass& x, const DevPass& y) {
  return std::memcmp(x.tma_kind, y.tma_kind, sizeof(x.tma_kind)) == 0 &&
         std::memcmp(x.tma_qlo, y.tma_qlo, sizeof(x.tma_qlo)) == 0 &&
         std::memcmp(x.tma_bits, y.tma_bits, sizeof(x.tma_bits)) == 0;
}

// Tensor maps for pass p over (buf0, buf1), encoded once per view and buffers.
const PassMaps* pass_maps_for(qml_ctx* c, const DevPass& dp, bool backward, int B, const void* buf0,
                              const void* buf1) {
  static const PassMaps none{};
  if (!dp.tma || !buf0) return &none;
  for (const qml_ctx::MapEntry& m : c->maps)
    if (m.backward == backward && m.B == B && m.buf0 == buf0 && m.buf1 == buf1 && same_tma_view(m.view, dp))
      return &m.maps;
  qml_ctx::MapEntry m{};
  m.view = dp, m.backward = backward, m.B = B, m.buf0 = buf0, m.buf1 = buf1;
  if (encode_pass_maps(dp, c->cfg.n_qubits, B, backward, buf0, buf1, &m.maps) != cudaSuccess) return nullptr;
  // A plan has a few tile views, and a call rotates through at most three
  // buffers (the CNOT gather's backward: psi, lambda, scratch), so the
  // entries in use number at most views x 6 ordered buffer pairs x 2
  // directions per batch size: well under the cap, which only bounds a
  // context that sees many different buffers.
  if (c->maps.size() >= 256) c->maps.clear();
  c->maps.push_back(m);
  return &c->maps.back().maps;
}

const PassMaps* pass_maps(qml_ctx* c, int p, bool backward, int B, const void* buf0, const void* buf1) {
  return pass_maps_for(c, fp32_passes(c)[p], backward, B, buf0, buf1);
}

// Copy the observable's terms into the workspace if they changed since the
// last upload (a copy from pageable host memory: it may wait for the stream).
cudaError_t upload_observable(qml_ctx* c, cudaStream_t s) {
  if (!c->obs_dirty || c->obs_terms.empty()) {
    c->obs_dirty = false;
    return cudaSuccess;
  }
  cudaError_t e = cudaMemcpyAsync(c->ws + c->lay.obs_groups, c->obs_groups.data(),
                                  sizeof(ObsGroup) * c->obs_groups.size(), cudaMemcpyHostToDevice, s);
  if (e == cudaSuccess)
    e = cudaMemcpyAsync(c->ws + c->lay.obs_terms, c->obs_terms.data(), sizeof(ObsTerm) * c->obs_terms.size(),
                        cudaMemcpyHostToDevice, s);
  if (e == cudaSuccess) c->obs_dirty = false;
  return e;
}

cudaError_t launch_expectation(qml_ctx* c, const float2* psi, int B, float* expect, cudaStream_t s) {
  const int n = c->cfg.n_qubits;
  if (c->obs_terms.empty())
    return launch_expect(psi, B, n, at<double>(c, c->lay.exp_partial), expect, at<unsigned>(c, c->lay.status), s);
  cudaError_t e = upload_observable(c, s);
  if (e != cudaSuccess) return e;
  return launch_obs_expect(psi, B, n, at<ObsGroup>(c, c->lay.obs_groups), (int)c->obs_groups.size(),
                           at<ObsTerm>(c, c->lay.obs_terms), at<double>(c, c->lay.exp_partial), expect,
                           at<unsigned>(c, c->lay.status), s);
}

// Neighbour masks of the entangler (a bond listed twice cancels).
void set_bond_masks(qml_ctx* c) {
  for (int q = 0; q < kMaxQubits; ++q) c->nb[q] = c->nbhi[q] = 0;
  for (const auto& e : c->bonds) {
    c->nb[e.first] ^= 1u << e.second;
    c->nb[e.second] ^= 1u << e.first;
    c->nbhi[std::min(e.first, e.second)] ^= 1u << std::max(e.first, e.second);
  }
}

// Conversion between the standard order and the working-state order of the
// plan (addr_of); both move only the lowest index bits, within chunks.
cudaError_t convert_layout(qml_ctx* c, float2* buf, int B, bool to_working, cudaStream_t s) {
  const int n = c->cfg.n_qubits;
  int cb = 0;
  for (int q = 0; q < n; ++q)
    if (c->plan.addr_of[q] != q) cb = std::max(cb, std::max(q, c->plan.addr_of[q]) + 1);
  if (cb == 0) return cudaSuccess;
  ++c->launches;
  int to[kTileBits];
  for (int b = 0; b < cb; ++b) {
    if (to_working) to[b] = c->plan.addr_of[b];  // standard bit b -> its address bit
    else
      for (int q = 0; q < cb; ++q)
        if (c->plan.addr_of[q] == b) to[b] = q;  // address bit b -> its qubit
  }
  return launch_permute_bits(buf, (long long)B << n, cb, to, c->sms, s);
}

// ------------------------------------------------------------ CNOT entanglers

// Upload the one-layer schedules (pageable host memory: the copy may wait
// for the stream) once per workspace layout.
cudaError_t upload_sub(qml_ctx* c, cudaStream_t s) {
  if (c->sub_uploaded) return cudaSuccess;
  const size_t P1 = c->sub[0].size();
  cudaError_t e = cudaSuccess;
  for (int v = 0; v < 4 && e == cudaSuccess; ++v)
    e = cudaMemcpyAsync(c->ws + c->lay.sub_passes + sizeof(DevPass) * P1 * v, c->sub[v].data(),
                        sizeof(DevPass) * P1, cudaMemcpyHostToDevice, s);
  std::vector<int> sp(c->plan1.slot_pass.begin(), c->plan1.slot_pass.end());
  std::vector<int> si(c->plan1.slot_index.begin(), c->plan1.slot_index.end());
  if (e == cudaSuccess)
    e = cudaMemcpyAsync(c->ws + c->lay.sub_slot_pass, sp.data(), sizeof(int) * sp.size(), cudaMemcpyHostToDevice, s);
  if (e == cudaSuccess)
    e = cudaMemcpyAsync(c->ws + c->lay.sub_slot_index, si.data(), sizeof(int) * si.size(), cudaMemcpyHostToDevice,
                        s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);  // the host vectors above are temporaries
  if (e == cudaSuccess) c->sub_uploaded = true;
  return e;
}

// Schedule variant of layer l: the first layer encodes, the last one leaves
// the standard layout.
int sub_variant(int l, int L) { return (l == 0 ? 2 : 0) + (l == L - 1 ? 1 : 0); }

qml_status run_forward_cnot(qml_ctx* c, const float* theta, const float* x, int B, float2* psi, float* expect,
                            cudaStream_t s) {
  c->prep_theta = nullptr;  // the per-layer tables below overwrite the prepared ones
  const int n = c->cfg.n_qubits, L = c->cfg.n_layers, cb = c->cfg.ckpt_block;
  if (c->ws_bytes < c->lay.base_total) return QML_ERR_WORKSPACE;
  cudaError_t e = upload_sub(c, s);
  if (e != cudaSuccess) return QML_ERR_CUDA;
  const int P1 = (int)c->sub[0].size();
  CoefRegion* cf = at<CoefRegion>(c, c->lay.coef_fwd);
  CoefRegion* ci = at<CoefRegion>(c, c->lay.coef_inv);
  e = launch_prep_enc(x, B, n, at<float2>(c, c->lay.enc), s);
  if (e != cudaSuccess) return QML_ERR_CUDA;
  PassArgs a{};
  a.region = c->region;
  a.n = n;
  a.B = B;
  a.U = (B + 1) / 2;
  a.N = c->N;
  a.enc = at<float2>(c, c->lay.enc);
  a.ckpt = c->ws + c->lay.ckpt;
  a.storage = c->cfg.storage == QML_STORE_BF16 ? 1 : 0;
  a.bmax = c->cfg.max_batch;
  a.status = at<unsigned>(c, c->lay.status);
  a.reupload = c->reupload ? 1 : 0;  // CZ neighbour masks stay zero: no CZ in this mode
  float2* cur = psi;
  float2* other = at<float2>(c, c->lay.scratch);
  float2* part = at<float2>(c, c->lay.dummy);  // partner plane of an odd batch's last unit
  float2* part_other = at<float2>(c, c->lay.dummy2);
  c->launches += 1;
  for (int l = 0; l < L; ++l) {
    const int v = sub_variant(l, L);
    const DevPass* dsub = at<DevPass>(c, c->lay.sub_passes) + (size_t)P1 * v;
    e = launch_prep_pass_coef(dsub, P1, theta + (size_t)l * n * 3, cf, ci, s);
    if (e == cudaSuccess && l == 0 && c->fault == qml_ctx::FAULT_NAN)  // injected: as in run_forward
      e = cudaMemsetAsync(cf, 0xff, sizeof(float4), s);
    if (e != cudaSuccess) return QML_ERR_CUDA;
    ++c->launches;
    qml_ctx::Span sp{};
    const bool timed = span_begin(c, s, &sp, false);
    for (int p = 0; p < P1; ++p) {
      const DevPass& dp = c->sub[v][p];
      a.n_tiles = (int)(((a.U + (1ll << dp.unit_bits) - 1) >> dp.unit_bits) << dp.n_out);
      a.buf0 = cur;
      a.dummy = part;
      const PassMaps* maps = pass_maps_for(c, dp, false, B, cur, part);
      if (!maps) return QML_ERR_CUDA;
      e = launch_pass(false, a, dp, *maps, c->grid_fwd, c->smem, s, cf + p);
      if (e != cudaSuccess) return QML_ERR_CUDA;
      ++c->launches;
    }
    if (timed) {
      sp.passes = P1;
      span_end(c, s, &sp);
    }
    // the layer's CNOT list: psi'(j) = psi(M^-1 j), on every plane
    e = launch_gather_bits(cur, other, n, B, c->cnot_fwd, c->cnot_bwd, c->sms, s);
    if (e == cudaSuccess && (B & 1) && l + 1 < L)
      e = launch_gather_bits(part, part_other, n, 1, c->cnot_fwd, c->cnot_bwd, c->sms, s);
    if (e != cudaSuccess) return QML_ERR_CUDA;
    c->launches += (B & 1) && l + 1 < L ? 2 : 1;
    std::swap(cur, other);
    std::swap(part, part_other);
    if (cb > 0 && (l + 1) % cb == 0 && l + 1 < L) {  // slot m holds the state after layer (m + 1) b - 1
      const int m = (l + 1) / cb - 1;
      void* slot = c->ws + c->lay.ckpt + slot_bytes(c) * (size_t)m * c->cfg.max_batch * (size_t)c->N;
      e = int8_slots(c) ? launch_slot8_from_planes(cur, part, slot8_codes(c, m), slot8_exps(c, m), B, n, s)
                        : launch_slot_from_planes(cur, part, slot, a.storage, B, n, c->sms, s);
      if (e != cudaSuccess) return QML_ERR_CUDA;
      ++c->launches;
      c->ckpt_batch[m] = B;
    }
  }
  if (cur != psi) {
    e = cudaMemcpyAsync(psi, cur, sizeof(float2) * (size_t)B * c->N, cudaMemcpyDeviceToDevice, s);
    if (e != cudaSuccess) return QML_ERR_CUDA;
  }
  e = convert_layout(c, psi, B, false, s);  // working-state order -> standard order (three or more sets)
  if (e != cudaSuccess) return QML_ERR_CUDA;
  if (expect) {
    c->launches += 2;
    e = launch_expectation(c, psi, B, expect, s);
    if (e != cudaSuccess) return QML_ERR_CUDA;
  }
  return QML_OK;
}

qml_status run_backward_cnot(qml_ctx* c, const float* theta, const float* x, int B, float2* psi, float2* lam,
                             const float* g, float* grad, cudaStream_t s) {
  c->prep_theta = nullptr;
  const int n = c->cfg.n_qubits, L = c->cfg.n_layers, cb = c->cfg.ckpt_block;
  if (c->ws_bytes < c->lay.base_total) return QML_ERR_WORKSPACE;
  for (int m = 0; m < c->plan.n_ckpt; ++m)
    if (c->ckpt_batch[m] != B) return QML_ERR_CKPT_MISMATCH;
  cudaError_t e = upload_sub(c, s);
  if (e != cudaSuccess) return QML_ERR_CUDA;
  const int P1 = (int)c->sub[0].size();
  CoefRegion* cf = at<CoefRegion>(c, c->lay.coef_fwd);
  CoefRegion* ci = at<CoefRegion>(c, c->lay.coef_inv);
  if (c->obs_terms.empty()) {
    e = launch_bwd_init(psi, lam, g, B, n, s);
  } else {
    e = upload_observable(c, s);
    if (e == cudaSuccess)
      e = launch_obs_bwd_init(psi, lam, g, B, n, at<ObsGroup>(c, c->lay.obs_groups), (int)c->obs_groups.size(),
                              at<ObsTerm>(c, c->lay.obs_terms), s);
  }
  if (e == cudaSuccess) e = convert_layout(c, psi, B, true, s);  // both planes: standard -> working order
  if (e == cudaSuccess) e = convert_layout(c, lam, B, true, s);
  if (e != cudaSuccess) return QML_ERR_CUDA;
  if (c->reupload) {
    e = launch_prep_enc(x, B, n, at<float2>(c, c->lay.enc), s);
    if (e != cudaSuccess) return QML_ERR_CUDA;
  }
  PassArgs a{};
  a.region = c->region;
  a.n = n;
  a.B = B;
  a.U = B;
  a.N = c->N;
  a.enc = at<float2>(c, c->lay.enc);
  a.g = g;
  a.ckpt = c->ws + c->lay.ckpt;
  a.storage = c->cfg.storage == QML_STORE_BF16 ? 1 : 0;
  a.bmax = c->cfg.max_batch;
  a.partials = at<float>(c, c->lay.partials);
  a.status = at<unsigned>(c, c->lay.status);
  a.reupload = c->reupload ? 1 : 0;
  float2* b0 = psi;  // plane 0: (Re psi, Re lambda)
  float2* b1 = lam;  // plane 1: (Im psi, Im lambda)
  float2* sc = at<float2>(c, c->lay.scratch);
  c->launches += 1;
  for (int l = L - 1; l >= 0; --l) {
    if (cb > 0 && (l + 1) % cb == 0 && l + 1 < L) {  // the stored state after layer l replaces the uncomputed one
      const int m = (l + 1) / cb - 1;
      const void* slot = c->ws + c->lay.ckpt + slot_bytes(c) * (size_t)m * c->cfg.max_batch * (size_t)c->N;
      e = int8_slots(c)
              ? launch_slot8_to_planes(b0, b1, slot8_codes(c, m), slot8_exps(c, m), nullptr, B, n, s)
              : launch_restore_planes(b0, b1, slot, a.storage, (long long)B * c->N, c->sms, s);
      if (e != cudaSuccess) return QML_ERR_CUDA;
      ++c->launches;
    }
    // un-apply the layer's CNOT list: psi(b) = psi'(M b), on both planes
    e = launch_gather_bits(b0, sc, n, B, c->cnot_bwd, c->cnot_fwd, c->sms, s);
    if (e != cudaSuccess) return QML_ERR_CUDA;
    std::swap(b0, sc);
    e = launch_gather_bits(b1, sc, n, B, c->cnot_bwd, c->cnot_fwd, c->sms, s);
    if (e != cudaSuccess) return QML_ERR_CUDA;
    std::swap(b1, sc);
    c->launches += 2;
    const int v = sub_variant(l, L);
    const DevPass* dsub = at<DevPass>(c, c->lay.sub_passes) + (size_t)P1 * v;
    e = launch_prep_pass_coef(dsub, P1, theta + (size_t)l * n * 3, cf, ci, s);
    if (e != cudaSuccess) return QML_ERR_CUDA;
    ++c->launches;
    qml_ctx::Span sp{};
    const bool timed = span_begin(c, s, &sp, true);
    for (int p = P1 - 1; p >= 0; --p) {
      const DevPass& dp = c->sub[v][p];
      a.n_tiles = (int)(((a.U + (1ll << dp.unit_bits) - 1) >> dp.unit_bits) << dp.n_out);
      a.buf0 = b0;
      a.buf1 = b1;
      const PassMaps* maps = pass_maps_for(c, dp, true, B, b0, b1);
      if (!maps) return QML_ERR_CUDA;
      e = launch_pass(true, a, dp, *maps, c->grid_bwd, c->smem, s, ci + p);
      if (e != cudaSuccess) return QML_ERR_CUDA;
      ++c->launches;
    }
    if (timed) {
      sp.passes = P1;
      span_end(c, s, &sp);
    }
    e = launch_grad_reduce(dsub, at<int>(c, c->lay.sub_slot_pass), at<int>(c, c->lay.sub_slot_index),
                           at<float>(c, c->lay.partials), c->grid_bwd, theta + (size_t)l * n * 3, nullptr, 1, n,
                           grad + (size_t)l * n * 3, at<unsigned>(c, c->lay.status), s);
    if (e != cudaSuccess) return QML_ERR_CUDA;
    ++c->launches;
  }
  return QML_OK;
}

// Coefficient tables of the fp32 passes from theta (both directions).
cudaError_t prep_coefficients(qml_ctx* c, const float* theta, cudaStream_t s) {
  CoefRegion* cf = at<CoefRegion>(c, c->lay.coef_fwd);
  CoefRegion* ci = at<CoefRegion>(c, c->lay.coef_inv);
  if (!use_split(c))
    return launch_prep_pass_coef(at<DevPass>(c, c->lay.passes), (int)c->dpass.size(), theta, cf, ci, s);
  if (c->cnot) {  // the fused CNOT schedule: one segment per layer and qubit set
    uint32_t set0 = 0;
    for (int q : c->plan.sets[0]) set0 |= 1u << q;
    return launch_prep_split_cnot(at<DevPass>(c, c->lay.passes_split), (int)c->dpass_split.size(), theta,
                                  c->cfg.n_layers, c->cfg.n_qubits, set0, at<int>(c, c->lay.undo),
                                  at<SplitRot>(c, c->lay.s_rot), at<SplitLayer>(c, c->lay.s_lay),
                                  at<double>(c, c->lay.s_gfix), at<float2>(c, c->lay.s_dqf),
                                  at<float2>(c, c->lay.s_dqb), cf, ci, at<float>(c, c->lay.rscale), s);
  }
  return launch_prep_split(at<DevPass>(c, c->lay.passes_split), (int)c->dpass_split.size(), theta,
                           c->cfg.n_layers, c->cfg.n_qubits, at<int>(c, c->lay.undo), at<SplitRot>(c, c->lay.s_rot),
                           at<SplitLayer>(c, c->lay.s_lay), at<double>(c, c->lay.s_gfix),
                           at<float2>(c, c->lay.s_dqf), at<float2>(c, c->lay.s_dqb), cf, ci,
                           at<float>(c, c->lay.rscale), s);
}

// Kernel launches of prep_coefficients.
int prep_launches(const qml_ctx* c) {
  if (!use_split(c)) return 1;
  if (c->cnot) return 4;
  return prep_split_launches(c->cfg.n_layers, c->cfg.n_qubits, (int)c->dpass_split.size());
}

// A pass that neither writes nor restores its slot (8-bit slots).
DevPass without_slot(const DevPass& dp) {
  DevPass q = dp;
  q.ckpt = -1;
  return q;
}

qml_status run_forward(qml_ctx* c, const float* theta, const float* x, int B, float2* psi,
                       float* expect, cudaStream_t s) {
  if (c->cnot && !cnot_fused_now(c)) return run_forward_cnot(c, theta, x, B, psi, expect, s);
  const int n = c->cfg.n_qubits;
  const bool split = use_split(c);
  const std::vector<DevPass>& passes = fp32_passes(c);
  const int P = (int)passes.size();
  CoefRegion* cf = at<CoefRegion>(c, c->lay.coef_fwd);
  cudaError_t e = prep_coefficients(c, theta, s);
  c->prep_theta = e == cudaSuccess ? theta : nullptr;
  c->prep_gen = c->gen;
  if (e == cudaSuccess && c->fault == qml_ctx::FAULT_NAN)  // injected: the first rotation's coefficients become NaN
    e = cudaMemsetAsync(cf, 0xff, sizeof(float4), s);
  if (e != cudaSuccess) return QML_ERR_CUDA;
  e = launch_prep_enc(x, B, n, at<float2>(c, c->lay.enc), s);
  if (e != cudaSuccess) return QML_ERR_CUDA;
  PassArgs a{};
  a.region = c->region;
  a.n = n;
  a.B = B;
  a.U = (B + 1) / 2;
  a.N = c->N;
  a.buf0 = psi;
  a.buf1 = nullptr;
  a.dummy = at<float2>(c, c->lay.dummy);
  a.enc = at<float2>(c, c->lay.enc);
  a.g = nullptr;
  a.ckpt = c->ws + c->lay.ckpt;
  a.storage = c->cfg.storage == QML_STORE_BF16 ? 1 : 0;
  a.bmax = c->cfg.max_batch;
  a.partials = nullptr;
  a.status = at<unsigned>(c, c->lay.status);
  for (int q = 0; q < kMaxQubits; ++q) a.cz_nb[q] = c->cnot ? 0u : c->nb[q], a.cz_nbhi[q] = c->cnot ? 0u : c->nbhi[q];
  a.reupload = c->reupload ? 1 : 0;
  a.dq = split ? at<float2>(c, c->lay.s_dqf) : nullptr;
  a.rscale = nullptr;
  // Z0 from the last pass's registers (tiles of one batch unit): per tile
  // partials, then one fixed-order sum per sample
  const bool epi = expect && fused_z0(c) && passes[P - 1].unit_bits == 0;
  a.epart = epi ? at<double>(c, c->lay.exp_partial) : nullptr;
  c->launches += prep_launches(c) + 1;  // coefficient prep, encoding table
  qml_ctx::Span sp{};
  const bool timed = span_begin(c, s, &sp, false);
  if (split && !passes[0].tma) {  // one tile holds the state: every pass in one launch
    const DevPass& dp = passes[0];
    // One sample per batch unit with the amplitude in a lane pair (half the
    // work per tile of the two-sample form) for the chain from the encoding
    // to the standard order, CZ entanglers: taken where it gives more tiles
    // than the two-sample form (a tile of one batch unit, or batches that
    // fill more than one tile), not for the single tile of a small batch.
    const long long upt = 1ll << dp.unit_bits;
    const bool more_tiles = (B + upt - 1) / upt > (a.U + upt - 1) / upt;
    a.zf = (passes[0].gen && passes[P - 1].last && !c->cnot && !dp.slow && more_tiles) ? 1 : 0;
    if (a.zf) a.U = B;
    a.npass = P;
    a.passes = at<DevPass>(c, c->lay.passes_split);
    a.coef = cf;
    a.n_tiles = (int)(((a.U + (1ll << dp.unit_bits) - 1) >> dp.unit_bits) << dp.n_out);
    static const PassMaps none{};
    e = launch_pass(false, a, dp, none, c->grid_fwd, c->smem_multi, s);
    if (e != cudaSuccess) return QML_ERR_CUDA;
    ++c->launches;
    sp.passes = 1;  // the span times one launch
    for (const DevPass& q : passes)
      if (q.ckpt >= 0) c->ckpt_batch[q.ckpt] = B;
  }
  for (int p = 0; p < P && !(split && !passes[0].tma); ++p) {
    const DevPass& dp = passes[p];
    const long long units_per_tile = 1ll << dp.unit_bits;
    a.n_tiles = (int)(((a.U + units_per_tile - 1) / units_per_tile) << dp.n_out);
    const PassMaps* maps = pass_maps(c, p, false, B, psi, a.dummy);
    if (!maps) return QML_ERR_CUDA;
    const bool slot8 = int8_slots(c) && dp.ckpt >= 0;
    e = launch_pass(false, a, slot8 ? without_slot(dp) : dp, *maps, c->grid_fwd, c->smem, s, cf + p);
    if (e == cudaSuccess && slot8) {
      e = launch_slot8_from_planes(psi, a.dummy, slot8_codes(c, dp.ckpt), slot8_exps(c, dp.ckpt), B, n, s);
      ++c->launches;
    }
    if (e != cudaSuccess) return QML_ERR_CUDA;
    ++c->launches;
    if (dp.ckpt >= 0) c->ckpt_batch[dp.ckpt] = B;
  }
  if (c->fault == qml_ctx::FAULT_CKPT) std::fill(c->ckpt_batch.begin(), c->ckpt_batch.end(), -1);  // injected
  if (timed) span_end(c, s, &sp);
  e = convert_layout(c, psi, B, false, s);  // working-state order -> standard order
  if (e != cudaSuccess) return QML_ERR_CUDA;
  if (epi) {
    c->launches += 1;
    const int tps = 1 << (n > kTileBits ? n - kTileBits : 0);  // tiles per sample
    e = launch_expect_final(at<double>(c, c->lay.exp_partial), tps, B, expect, at<unsigned>(c, c->lay.status), s);
    if (e != cudaSuccess) return QML_ERR_CUDA;
  } else if (expect) {
    c->launches += 2;
    e = launch_expectation(c, psi, B, expect, s);
    if (e != cudaSuccess) return QML_ERR_CUDA;
  }
  return QML_OK;
}

qml_status run_backward(qml_ctx* c, const float* theta, const float* x, int B, float2* psi,
                        float2* lam, const float* g, float* grad, cudaStream_t s) {
  if (c->cnot && !cnot_fused_now(c)) return run_backward_cnot(c, theta, x, B, psi, lam, g, grad, s);
  const int n = c->cfg.n_qubits, L = c->cfg.n_layers;
  const bool split = use_split(c);
  const std::vector<DevPass>& passes = fp32_passes(c);
  const int P = (int)passes.size();
  for (int m = 0; m < c->plan.n_ckpt; ++m)
    if (c->ckpt_batch[m] != B) return QML_ERR_CKPT_MISMATCH;
  CoefRegion* ci = at<CoefRegion>(c, c->lay.coef_inv);
  // the forward call that produced psi prepared the tables of both
  // directions from the same theta: reuse them
  const bool reuse = c->prep_theta == theta && c->prep_gen == c->gen;
  cudaError_t e = reuse ? cudaSuccess : prep_coefficients(c, theta, s);
  if (e != cudaSuccess) return QML_ERR_CUDA;
  if (reuse) c->launches -= prep_launches(c);
  if (c->obs_terms.empty()) {
    e = launch_bwd_init(psi, lam, g, B, n, s);
  } else {
    e = upload_observable(c, s);
    if (e == cudaSuccess)
      e = launch_obs_bwd_init(psi, lam, g, B, n, at<ObsGroup>(c, c->lay.obs_groups), (int)c->obs_groups.size(),
                              at<ObsTerm>(c, c->lay.obs_terms), s);
  }
  if (e != cudaSuccess) return QML_ERR_CUDA;
  e = convert_layout(c, psi, B, true, s);  // both backward planes: standard -> working-state order
  if (e == cudaSuccess) e = convert_layout(c, lam, B, true, s);
  if (e != cudaSuccess) return QML_ERR_CUDA;
  if (c->reupload) {  // per-sample encoding angles for un-applying the re-uploaded encodings
    e = launch_prep_enc(x, B, n, at<float2>(c, c->lay.enc), s);
    if (e != cudaSuccess) return QML_ERR_CUDA;
  }
  PassArgs a{};
  a.region = c->region;
  a.n = n;
  a.B = B;
  a.U = B;
  a.N = c->N;
  a.buf0 = psi;
  a.buf1 = lam;
  a.dummy = nullptr;
  a.enc = at<float2>(c, c->lay.enc);
  a.g = g;
  a.ckpt = c->ws + c->lay.ckpt;
  a.storage = c->cfg.storage == QML_STORE_BF16 ? 1 : 0;
  a.bmax = c->cfg.max_batch;
  a.partials = at<float>(c, c->lay.partials);
  a.status = at<unsigned>(c, c->lay.status);
  for (int q = 0; q < kMaxQubits; ++q) a.cz_nb[q] = c->cnot ? 0u : c->nb[q], a.cz_nbhi[q] = c->cnot ? 0u : c->nbhi[q];
  a.reupload = c->reupload ? 1 : 0;
  a.dq = split ? at<float2>(c, c->lay.s_dqb) : nullptr;
  c->launches += prep_launches(c) + 2;  // coefficient prep, lambda init, gradient reduce
  qml_ctx::Span sp{};
  const bool timed = span_begin(c, s, &sp, true);
  const bool one_launch = split && !passes[0].tma;  // one tile holds the state: every pass in one launch
  if (one_launch) {
    const DevPass& dp = passes[0];
    a.npass = P;
    a.passes = at<DevPass>(c, c->lay.passes_split);
    a.coef = ci;
    a.rscale = at<float>(c, c->lay.rscale);
    a.n_tiles = (int)(((a.U + (1ll << dp.unit_bits) - 1) >> dp.unit_bits) << dp.n_out);
    static const PassMaps none{};
    e = launch_pass(true, a, dp, none, c->grid_bwd, c->smem_multi, s);
    if (e != cudaSuccess) return QML_ERR_CUDA;
    ++c->launches;
    sp.passes = 1;  // the span times one launch
  }
  for (int p = P - 1; p >= 0 && !one_launch; --p) {
    const DevPass& dp = passes[p];
    const long long units_per_tile = 1ll << dp.unit_bits;
    a.n_tiles = (int)(((a.U + units_per_tile - 1) / units_per_tile) << dp.n_out);
    a.rscale = (split && dp.ckpt >= 0) ? at<float>(c, c->lay.rscale) + p : nullptr;
    const PassMaps* maps = pass_maps(c, p, true, B, psi, lam);
    if (!maps) return QML_ERR_CUDA;
    const bool slot8 = int8_slots(c) && dp.ckpt >= 0;
    if (slot8) {
      e = launch_slot8_to_planes(psi, lam, slot8_codes(c, dp.ckpt), slot8_exps(c, dp.ckpt), a.rscale, B, n, s);
      if (e != cudaSuccess) return QML_ERR_CUDA;
      ++c->launches;
    }
    e = launch_pass(true, a, slot8 ? without_slot(dp) : dp, *maps, c->grid_bwd, c->smem, s, ci + p);
    if (e != cudaSuccess) return QML_ERR_CUDA;
    ++c->launches;
  }
  if (timed) span_end(c, s, &sp);
  e = launch_grad_reduce(at<DevPass>(c, c->lay.passes), at<int>(c, c->lay.slot_pass),
                         at<int>(c, c->lay.slot_index), at<float>(c, c->lay.partials), c->grid_bwd,
                         theta, split ? at<double>(c, c->lay.s_gfix) : nullptr, L, n, grad,
                         at<unsigned>(c, c->lay.status), s);
  return cuda_status(e);
}

// fp64 tiles: the schedule's tile qubits, less the highest qubit the pass
// does not rotate when the tile has 12 (2^11-position tiles let two blocks
// share an SM; a passive qubit can leave the tile because CZ is diagonal).
uint32_t f64_tile_mask(const DevPass& dp, int n, uint32_t kept = 0) {
  uint32_t m = 0, rot = kept;
  for (int b = 0; b < kTileBits; ++b)
    if (dp.tile_q[b] >= 0 && dp.tile_q[b] < n) m |= 1u << dp.tile_q[b];
  for (int s = 0; s < dp.nslots; ++s) rot |= 1u << (dp.slot_lq[s] % n);
  const uint32_t passive = m & ~rot;
  if (__builtin_popcount(m) == kTileBits && passive) m &= ~(1u << (31 - __builtin_clz(passive)));
  return m;
}

void set_f64_tiles(qml_ctx* c) {
  const int n = c->cfg.n_qubits;
  c->f64_mask.clear();
  c->f64_tmax = 1;
  for (const DevPass& dp : c->dpass) {
    // fused CNOT layers: the set a pass's permutation changes stays in its tile
    uint32_t kept = 0;
    for (int o = 0; o < dp.nops; ++o)
      if (dp.ops[o].kind == OP_PERM)
        for (int q : c->plan.sets[dp.ops[o].c]) kept |= 1u << q;
    const uint32_t m = f64_tile_mask(dp, n, kept);
    c->f64_mask.push_back(m);
    c->f64_tmax = std::max(c->f64_tmax, __builtin_popcount(m));
  }
}

Pass64Args pass64_args(qml_ctx* c, const double* theta, const double* x, int B, double2* psi, double2* lam) {
  Pass64Args a{};
  const int n = c->cfg.n_qubits;
  a.n = n;
  a.B = B;
  a.tmax = c->f64_tmax;
  a.theta = theta;
  a.x = x;
  a.psi = psi;
  a.lam = lam;
  a.ckpt = c->ws + c->lay.ckpt;
  a.storage = c->cfg.storage == QML_STORE_FP64 ? 2 : c->cfg.storage == QML_STORE_BF16 ? 1 : 0;
  a.slot_elems = (long long)c->cfg.max_batch * c->N;
  a.partials = at<double>(c, c->lay.partials);
  a.status = at<unsigned>(c, c->lay.status);
  a.reupload = c->reupload ? 1 : 0;
  for (int q = 0; q < kMaxQubits; ++q) a.nb[q] = c->cnot ? 0u : c->nb[q], a.nbhi[q] = c->cnot ? 0u : c->nbhi[q];
  a.L = c->cfg.n_layers;
  if (c->cnot_fused)
    for (int g = 0; g < 2; ++g)
      for (int q = 0; q < kMaxQubits; ++q) a.perm_fwd[g][q] = c->cnot_map.inv[g][q], a.perm_bwd[g][q] = c->cnot_map.fwd[g][q];
  if (use_split64(c)) {
    a.srot = at<SplitRot>(c, c->lay.s_rot);
    a.slay = at<SplitLayer>(c, c->lay.s_lay);
  }
  return a;
}

// Split-form tables of an fp64 context from theta (both directions).
cudaError_t prep_split64(qml_ctx* c, const double* theta, cudaStream_t s) {
  c->launches += 4;
  return launch_prep_split64(at<DevPass>(c, c->lay.passes_split), (int)c->dpass_split.size(), theta,
                             c->cfg.n_layers, c->cfg.n_qubits, at<int>(c, c->lay.undo),
                             at<SplitRot>(c, c->lay.s_rot), at<SplitLayer>(c, c->lay.s_lay),
                             at<double>(c, c->lay.s_gfix), at<double2>(c, c->lay.s_dq64f),
                             at<double2>(c, c->lay.s_dq64b), at<double>(c, c->lay.rscale64), s);
}

void set_pass_tile(const qml_ctx* c, int p, int B, Pass64Args* a) {
  a->tile_mask = c->f64_mask[p];
  a->T = __builtin_popcount(a->tile_mask);
  a->n_tiles = (long long)B << (c->cfg.n_qubits - a->T);
}

void set_sub_tile(const qml_ctx* c, int p, int B, Pass64Args* a) {
  a->tile_mask = c->sub_mask[p];
  a->T = __builtin_popcount(a->tile_mask);
  a->n_tiles = (long long)B << (c->cfg.n_qubits - a->T);
}

// fp64 with CNOT entanglers: the one-layer passes, then the layer's CNOT
// list as a permutation of the standard-order state (qubit-bit maps).
qml_status run_forward64_cnot(qml_ctx* c, const double* theta, const double* x, int B, double2* psi,
                              double* expect, cudaStream_t s);
qml_status run_backward64_cnot(qml_ctx* c, const double* theta, const double* x, int B, double2* psi,
                               double2* lam, const double* g, double* grad, cudaStream_t s);

// E = <psi|O|psi> in fp64 (O = Z0 or the Pauli sum in force).
cudaError_t expect64(qml_ctx* c, const double2* psi, int B, double* expect, cudaStream_t s) {
  c->launches += 2;
  if (c->obs_terms.empty())
    return launch_expect64(psi, B, c->cfg.n_qubits, at<double>(c, c->lay.exp_partial), expect,
                           at<unsigned>(c, c->lay.status), s);
  cudaError_t e = upload_observable(c, s);
  if (e != cudaSuccess) return e;
  return launch_obs_expect64(psi, B, c->cfg.n_qubits, at<ObsGroup>(c, c->lay.obs_groups), (int)c->obs_groups.size(),
                             at<ObsTerm>(c, c->lay.obs_terms), at<double>(c, c->lay.exp_partial), expect,
                             at<unsigned>(c, c->lay.status), s);
}

// lambda = g O psi in fp64.
cudaError_t seed64(qml_ctx* c, const double2* psi, double2* lam, const double* g, int B, cudaStream_t s) {
  ++c->launches;
  if (c->obs_terms.empty()) return launch_bwd_init64(psi, lam, g, B, c->cfg.n_qubits, s);
  cudaError_t e = upload_observable(c, s);
  if (e != cudaSuccess) return e;
  return launch_obs_bwd_init64(psi, lam, g, B, c->cfg.n_qubits, at<ObsGroup>(c, c->lay.obs_groups),
                               (int)c->obs_groups.size(), at<ObsTerm>(c, c->lay.obs_terms), s);
}

qml_status run_forward64_cnot(qml_ctx* c, const double* theta, const double* x, int B, double2* psi,
                              double* expect, cudaStream_t s) {
  const int n = c->cfg.n_qubits, L = c->cfg.n_layers, cb = c->cfg.ckpt_block;
  if (c->ws_bytes < c->lay.base_total) return QML_ERR_WORKSPACE;
  cudaError_t e = upload_sub(c, s);
  if (e != cudaSuccess) return QML_ERR_CUDA;
  const int P1 = (int)c->sub[0].size();
  Pass64Args a = pass64_args(c, theta, x, B, psi, nullptr);
  for (int q = 0; q < kMaxQubits; ++q) a.nb[q] = a.nbhi[q] = 0;  // no CZ in this mode
  double2* cur = psi;
  double2* other = at<double2>(c, c->lay.scratch);
  for (int l = 0; l < L; ++l) {
    const int v = sub_variant(l, L);
    a.theta = theta + (size_t)l * n * 3;  // the one-layer passes read layer 0 of this pointer
    a.psi = cur;
    qml_ctx::Span sp{};
    const bool timed = span_begin(c, s, &sp, false);
    for (int p = 0; p < P1; ++p) {
      set_sub_tile(c, p, B, &a);
      if (launch_pass64(false, a, c->sub[v][p], (int)std::min<long long>(c->grid_fwd, a.n_tiles), s) != cudaSuccess)
        return QML_ERR_CUDA;
      ++c->launches;
    }
    if (timed) {
      sp.passes = P1;
      span_end(c, s, &sp);
    }
    e = launch_gather_bits64(cur, other, n, B, c->cnot_fwd_q, c->cnot_bwd_q, c->sms, s);
    if (e != cudaSuccess) return QML_ERR_CUDA;
    ++c->launches;
    std::swap(cur, other);
    if (cb > 0 && (l + 1) % cb == 0 && l + 1 < L) {
      const int m = (l + 1) / cb - 1;
      void* slot = c->ws + c->lay.ckpt + slot_bytes(c) * (size_t)m * c->cfg.max_batch * (size_t)c->N;
      e = launch_slot_copy64(true, cur, slot, a.storage, (long long)B * c->N, c->sms, s);
      if (e != cudaSuccess) return QML_ERR_CUDA;
      ++c->launches;
      c->ckpt_batch[m] = B;
    }
  }
  if (cur != psi) {
    e = cudaMemcpyAsync(psi, cur, sizeof(double2) * (size_t)B * c->N, cudaMemcpyDeviceToDevice, s);
    if (e != cudaSuccess) return QML_ERR_CUDA;
  }
  if (expect && expect64(c, psi, B, expect, s) != cudaSuccess) return QML_ERR_CUDA;
  return QML_OK;
}

qml_status run_backward64_cnot(qml_ctx* c, const double* theta, const double* x, int B, double2* psi,
                               double2* lam, const double* g, double* grad, cudaStream_t s) {
  const int n = c->cfg.n_qubits, L = c->cfg.n_layers, cb = c->cfg.ckpt_block;
  if (c->ws_bytes < c->lay.base_total) return QML_ERR_WORKSPACE;
  for (int m = 0; m < c->plan.n_ckpt; ++m)
    if (c->ckpt_batch[m] != B) return QML_ERR_CKPT_MISMATCH;
  cudaError_t e = upload_sub(c, s);
  if (e == cudaSuccess) e = seed64(c, psi, lam, g, B, s);
  if (e != cudaSuccess) return QML_ERR_CUDA;
  const int P1 = (int)c->sub[0].size();
  Pass64Args a = pass64_args(c, theta, x, B, psi, lam);
  for (int q = 0; q < kMaxQubits; ++q) a.nb[q] = a.nbhi[q] = 0;
  double2* b0 = psi;
  double2* b1 = lam;
  double2* sc = at<double2>(c, c->lay.scratch);
  for (int l = L - 1; l >= 0; --l) {
    if (cb > 0 && (l + 1) % cb == 0 && l + 1 < L) {  // the stored state after layer l replaces the uncomputed one
      const int m = (l + 1) / cb - 1;
      void* slot = c->ws + c->lay.ckpt + slot_bytes(c) * (size_t)m * c->cfg.max_batch * (size_t)c->N;
      e = launch_slot_copy64(false, b0, slot, a.storage, (long long)B * c->N, c->sms, s);
      if (e != cudaSuccess) return QML_ERR_CUDA;
      ++c->launches;
    }
    e = launch_gather_bits64(b0, sc, n, B, c->cnot_bwd_q, c->cnot_fwd_q, c->sms, s);
    if (e != cudaSuccess) return QML_ERR_CUDA;
    std::swap(b0, sc);
    e = launch_gather_bits64(b1, sc, n, B, c->cnot_bwd_q, c->cnot_fwd_q, c->sms, s);
    if (e != cudaSuccess) return QML_ERR_CUDA;
    std::swap(b1, sc);
    c->launches += 2;
    const int v = sub_variant(l, L);
    a.theta = theta + (size_t)l * n * 3;
    a.psi = b0;
    a.lam = b1;
    qml_ctx::Span sp{};
    const bool timed = span_begin(c, s, &sp, true);
    for (int p = P1 - 1; p >= 0; --p) {
      set_sub_tile(c, p, B, &a);
      if (launch_pass64(true, a, c->sub[v][p], c->grid_bwd, s) != cudaSuccess) return QML_ERR_CUDA;
      ++c->launches;
    }
    if (timed) {
      sp.passes = P1;
      span_end(c, s, &sp);
    }
    const DevPass* dsub = at<DevPass>(c, c->lay.sub_passes) + (size_t)P1 * v;
    e = launch_grad_reduce64(dsub, at<int>(c, c->lay.sub_slot_pass), at<int>(c, c->lay.sub_slot_index),
                             at<double>(c, c->lay.partials), c->grid_bwd, theta + (size_t)l * n * 3, nullptr, 1,
                             n, grad + (size_t)l * n * 3, at<unsigned>(c, c->lay.status), s);
    if (e != cudaSuccess) return QML_ERR_CUDA;
    ++c->launches;
  }
  return QML_OK;
}

qml_status run_forward64(qml_ctx* c, const double* theta, const double* x, int B, double2* psi, double* expect,
                         cudaStream_t s) {
  if (c->cnot && !cnot_fused_now(c)) return run_forward64_cnot(c, theta, x, B, psi, expect, s);
  Pass64Args a = pass64_args(c, theta, x, B, psi, nullptr);
  const bool split = use_split64(c);
  if (split) {
    if (prep_split64(c, theta, s) != cudaSuccess) return QML_ERR_CUDA;
    a.dq = at<double2>(c, c->lay.s_dq64f);
  }
  const std::vector<DevPass>& passes = split ? c->dpass_split : c->dpass;
  qml_ctx::Span sp{};
  const bool timed = span_begin(c, s, &sp, false);
  for (int p = 0; p < (int)passes.size(); ++p) {
    const DevPass& dp = passes[p];
    set_pass_tile(c, p, B, &a);
    if (launch_pass64(false, a, dp, (int)std::min<long long>(c->grid_fwd, a.n_tiles), s) != cudaSuccess)
      return QML_ERR_CUDA;
    ++c->launches;
    if (dp.ckpt >= 0) c->ckpt_batch[dp.ckpt] = B;
  }
  if (timed) span_end(c, s, &sp);
  if (expect && expect64(c, psi, B, expect, s) != cudaSuccess) return QML_ERR_CUDA;
  return QML_OK;
}

qml_status run_backward64(qml_ctx* c, const double* theta, const double* x, int B, double2* psi, double2* lam,
                          const double* g, double* grad, cudaStream_t s) {
  if (c->cnot && !cnot_fused_now(c)) return run_backward64_cnot(c, theta, x, B, psi, lam, g, grad, s);
  const int n = c->cfg.n_qubits, L = c->cfg.n_layers;
  for (int m = 0; m < c->plan.n_ckpt; ++m)
    if (c->ckpt_batch[m] != B) return QML_ERR_CKPT_MISMATCH;
  if (seed64(c, psi, lam, g, B, s) != cudaSuccess) return QML_ERR_CUDA;
  Pass64Args a = pass64_args(c, theta, x, B, psi, lam);
  const bool split = use_split64(c);
  if (split) {
    if (prep_split64(c, theta, s) != cudaSuccess) return QML_ERR_CUDA;
    a.dq = at<double2>(c, c->lay.s_dq64b);
  }
  const std::vector<DevPass>& passes = split ? c->dpass_split : c->dpass;
  ++c->launches;  // gradient reduce
  qml_ctx::Span sp{};
  const bool timed = span_begin(c, s, &sp, true);
  // every block writes its partials, so the grid is the one the layout counted
  for (int p = (int)passes.size() - 1; p >= 0; --p) {
    set_pass_tile(c, p, B, &a);
    a.rscale = (split && passes[p].ckpt >= 0) ? at<double>(c, c->lay.rscale64) + p : nullptr;
    if (launch_pass64(true, a, passes[p], c->grid_bwd, s) != cudaSuccess) return QML_ERR_CUDA;
    ++c->launches;
  }
  if (timed) span_end(c, s, &sp);
  return cuda_status(launch_grad_reduce64(at<DevPass>(c, c->lay.passes), at<int>(c, c->lay.slot_pass),
                                          at<int>(c, c->lay.slot_index), at<double>(c, c->lay.partials),
                                          c->grid_bwd, theta, split ? at<double>(c, c->lay.s_gfix) : nullptr, L, n,
                                          grad, at<unsigned>(c, c->lay.status), s));
}

}  // namespace

extern "C" {

int qml_abi_version(void) { return 1; }

const char* qml_status_str(qml_status s) {
  switch (s) {
    case QML_OK: return "ok";
    case QML_ERR_INVALID_ARG: return "invalid argument";
    case QML_ERR_UNSUPPORTED: return "unsupported configuration";
    case QML_ERR_WORKSPACE: return "workspace missing or too small";
    case QML_ERR_CUDA: return "CUDA runtime error";
    case QML_ERR_CKPT_MISMATCH: return "checkpoint slot mismatch";
    case QML_ERR_NUMERIC: return "non-finite value produced";
    case QML_ERR_BOUNDS: return "device bounds check failed";
    case QML_ERR_TIMEOUT: return "device wait timed out";
  }
  return "unknown status";
}

static qml_status create_ctx(const qml_config* cfg, int device, bool f64, qml_ctx** out);

qml_status qml_create(const qml_config* cfg, int device, qml_ctx** out) {
  if (cfg && cfg->storage == QML_STORE_FP64) {  // fp64 slots only for fp64 contexts
    if (out) *out = nullptr;
    return QML_ERR_INVALID_ARG;
  }
  return create_ctx(cfg, device, false, out);
}

qml_status qml_create_f64(const qml_config* cfg, int device, qml_ctx** out) {
  return create_ctx(cfg, device, true, out);
}

int qml_precision(const qml_ctx* c) { return c ? (c->f64 ? 64 : 32) : -1; }

static qml_status create_ctx(const qml_config* cfg, int device, bool f64, qml_ctx** out) {
  if (!out) return QML_ERR_INVALID_ARG;
  *out = nullptr;
  if (!cfg) return QML_ERR_INVALID_ARG;
  if (cfg->n_qubits < 1 || cfg->n_qubits > 30) return QML_ERR_INVALID_ARG;
  if (cfg->n_layers < 1 || cfg->n_layers > 100000) return QML_ERR_INVALID_ARG;
  if (cfg->max_batch < 1 || cfg->max_batch > (1 << 20)) return QML_ERR_INVALID_ARG;
  if (cfg->ckpt_block < 0) return QML_ERR_INVALID_ARG;
  if (cfg->storage != QML_STORE_FP32 && cfg->storage != QML_STORE_BF16 && cfg->storage != QML_STORE_FP64 &&
      cfg->storage != QML_STORE_INT8)
    return QML_ERR_INVALID_ARG;
  if (cfg->storage == QML_STORE_INT8 && f64) return QML_ERR_UNSUPPORTED;
  if (device < 0) return QML_ERR_INVALID_ARG;
  qml_ctx* c = new (std::nothrow) qml_ctx();
  if (!c) return QML_ERR_INVALID_ARG;
  c->cfg = *cfg;
  c->f64 = f64;
  if (const char* f = std::getenv("QML_FAULT")) {
    const std::string v(f);
    c->fault = v == "alloc" ? qml_ctx::FAULT_ALLOC
               : v == "ckpt_corrupt" ? qml_ctx::FAULT_CKPT
               : v == "nan_theta" ? qml_ctx::FAULT_NAN
                                  : qml_ctx::FAULT_NONE;
  }
  c->device = device;
  c->N = 1ll << cfg->n_qubits;
  std::string err = make_plan(cfg->n_qubits, cfg->n_layers, cfg->ckpt_block, &c->plan);
  if (!err.empty()) {
    delete c;
    return QML_ERR_UNSUPPORTED;
  }
  flatten_plan(c->plan, &c->dpass);
  flatten_plan(c->plan, &c->dpass_split, true);
  c->undo = undo_order(c->plan, c->dpass_split);
  c->bonds = chain_bonds(cfg->n_qubits);
  set_pass_entangler(c->plan, c->bonds, &c->dpass);
  set_pass_entangler(c->plan, c->bonds, &c->dpass_split);
  set_bond_masks(c);
  static std::atomic<int> next_region{0};
  c->region = next_region.fetch_add(1) % kCoefRegions;
  for (const DevPass& dp : c->dpass)
    if (dp.slow) c->slow = true;
  c->ckpt_batch.assign(c->plan.n_ckpt, -1);
  if (f64) set_f64_tiles(c);
  *out = c;
  return QML_OK;
}

qml_status qml_destroy(qml_ctx* ctx) {
  if (!ctx) return QML_ERR_INVALID_ARG;
  {
    DeviceGuard g(ctx->device);
    if (ctx->hg.exec) cudaGraphExecDestroy(ctx->hg.exec);
    if (ctx->cap) cudaStreamDestroy(ctx->cap);
  }
  for (auto& sp : ctx->spans) {
    cudaEventDestroy(sp.a);
    cudaEventDestroy(sp.b);
  }
  for (cudaEvent_t e : ctx->spare) cudaEventDestroy(e);
  delete ctx;
  return QML_OK;
}

size_t qml_workspace_bytes(const qml_ctx* cctx, int B) {
  qml_ctx* c = const_cast<qml_ctx*>(cctx);
  if (!c || B < 1 || B > c->cfg.max_batch) return 0;
  ensure_device(c);
  compute_layout(c);
  return c->lay.base_total;
}

size_t qml_host_workspace_bytes(const qml_ctx* cctx, int B) {
  qml_ctx* c = const_cast<qml_ctx*>(cctx);
  if (!c || B < 1 || B > c->cfg.max_batch) return 0;
  ensure_device(c);
  compute_layout(c);
  return c->lay.host_total;
}

qml_status qml_set_workspace(qml_ctx* c, void* ws, size_t bytes, void* stream) {
  if (!c || !ws) return QML_ERR_INVALID_ARG;
  ++c->gen;  // a captured host step no longer matches
  if (c->fault == qml_ctx::FAULT_ALLOC) return QML_ERR_WORKSPACE;  // injected: as if the buffer were too small
  if (misaligned(ws, kAlign)) return QML_ERR_INVALID_ARG;
  ensure_device(c);
  if (!c->dev_ok) return QML_ERR_CUDA;
  compute_layout(c);
  if (bytes < c->lay.base_total) return QML_ERR_WORKSPACE;
  DeviceGuard g(c->device);
  c->ws = static_cast<char*>(ws);
  c->ws_bytes = bytes;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  std::vector<int> sp(c->plan.slot_pass.begin(), c->plan.slot_pass.end());
  std::vector<int> si(c->plan.slot_index.begin(), c->plan.slot_index.end());
  cudaError_t e = cudaMemsetAsync(c->ws + c->lay.status, 0, 64, s);
  if (e == cudaSuccess)
    e = cudaMemcpyAsync(c->ws + c->lay.passes, c->dpass.data(), sizeof(DevPass) * c->dpass.size(),
                        cudaMemcpyHostToDevice, s);
  if (e == cudaSuccess)
    e = cudaMemcpyAsync(c->ws + c->lay.slot_pass, sp.data(), sizeof(int) * sp.size(), cudaMemcpyHostToDevice, s);
  if (e == cudaSuccess)
    e = cudaMemcpyAsync(c->ws + c->lay.slot_index, si.data(), sizeof(int) * si.size(), cudaMemcpyHostToDevice, s);
  if (e == cudaSuccess) e = cudaMemsetAsync(c->ws + c->lay.dummy, 0, sizeof(float2) * (size_t)c->N, s);
  if (e == cudaSuccess)
    e = cudaMemcpyAsync(c->ws + c->lay.passes_split, c->dpass_split.data(), sizeof(DevPass) * c->dpass_split.size(),
                        cudaMemcpyHostToDevice, s);
  if (e == cudaSuccess)
    e = cudaMemcpyAsync(c->ws + c->lay.undo, c->undo.data(), sizeof(int) * c->undo.size(), cudaMemcpyHostToDevice, s);
  // the host vectors above are pageable: the copies complete before return
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  std::fill(c->ckpt_batch.begin(), c->ckpt_batch.end(), -1);
  if (e != cudaSuccess) {
    c->ws = nullptr;
    return QML_ERR_CUDA;
  }
  return QML_OK;
}

qml_status qml_init_state_encode(qml_ctx* c, const float* x, int B, float* psi, void* stream) {
  qml_status st = check_ready(c, B);
  if (st != QML_OK) return st;
  if (!x || !psi || misaligned(psi, 8)) return QML_ERR_INVALID_ARG;
  DeviceGuard g(c->device);
  return cuda_status(launch_encode(x, B, c->cfg.n_qubits, reinterpret_cast<float2*>(psi),
                                   static_cast<cudaStream_t>(stream)));
}

qml_status qml_forward_expect(qml_ctx* c, const float* theta, const float* x, int B, float* psi,
                              float* expect, void* stream) {
  qml_status st = check_ready(c, B);
  if (st != QML_OK) return st;
  if (!theta || !x || !psi || !expect || misaligned(psi, 16)) return QML_ERR_INVALID_ARG;
  DeviceGuard g(c->device);
  return run_forward(c, theta, x, B, reinterpret_cast<float2*>(psi), expect, static_cast<cudaStream_t>(stream));
}

qml_status qml_backward_adjoint(qml_ctx* c, const float* theta, const float* x, int B, float* psi,
                                float* lambda, const float* dLdE, float* grad, void* stream) {
  qml_status st = check_ready(c, B);
  if (st != QML_OK) return st;
  if (!theta || !psi || !lambda || !dLdE || !grad || misaligned(psi, 16) || misaligned(lambda, 16))
    return QML_ERR_INVALID_ARG;
  if (psi == lambda) return QML_ERR_INVALID_ARG;
  if (c->reupload && !x) return QML_ERR_INVALID_ARG;  // the re-uploaded encodings need x
  DeviceGuard g(c->device);
  return run_backward(c, theta, x, B, reinterpret_cast<float2*>(psi), reinterpret_cast<float2*>(lambda),
                      dLdE, grad, static_cast<cudaStream_t>(stream));
}

qml_status qml_loss_seed(qml_ctx* c, const float* expect, const float* y, int B, float* g_out,
                         float* loss, void* stream) {
  qml_status st = check_ready(c, B);
  if (st != QML_OK) return st;
  if (!expect || !y) return QML_ERR_INVALID_ARG;
  DeviceGuard g(c->device);
  ++c->launches;
  return cuda_status(launch_loss_seed(expect, y, B, g_out, loss, static_cast<cudaStream_t>(stream)));
}

int qml_num_ckpt_slots(const qml_ctx* c) { return c ? c->plan.n_ckpt : -1; }

static qml_status ckpt_common(qml_ctx* c, int slot, const void* psi, int B) {
  qml_status st = check_ready(c, B);
  if (st != QML_OK) return st;
  if (!psi || misaligned(psi, 8)) return QML_ERR_INVALID_ARG;
  if (slot < 0 || slot >= c->plan.n_ckpt) return QML_ERR_INVALID_ARG;
  return QML_OK;
}

// 8-bit slots are in working-state order: the index bits of the addresses' lowest ones.
static cudaError_t copy_slot8(qml_ctx* c, bool save, int slot, float2* psi, int B, cudaStream_t s) {
  const int n = c->cfg.n_qubits;
  int cb = 0, to[kTileBits] = {};
  for (int q = 0; q < n; ++q)
    if (c->plan.addr_of[q] != q) cb = std::max(cb, std::max(q, c->plan.addr_of[q]) + 1);
  for (int q = 0; q < cb; ++q) to[c->plan.addr_of[q]] = q;
  ++c->launches;
  return launch_slot8_copy(save, psi, slot8_codes(c, slot), slot8_exps(c, slot), B, n, cb, to, s);
}

qml_status qml_ckpt_save(qml_ctx* c, int slot, const float* psi, int B, void* stream) {
  qml_status st = ckpt_common(c, slot, psi, B);
  if (st != QML_OK) return st;
  DeviceGuard g(c->device);
  if (int8_slots(c)) {
    if (copy_slot8(c, true, slot, reinterpret_cast<float2*>(const_cast<float*>(psi)), B,
                   static_cast<cudaStream_t>(stream)) != cudaSuccess)
      return QML_ERR_CUDA;
    c->ckpt_batch[slot] = B;
    return QML_OK;
  }
  const size_t elem = c->cfg.storage == QML_STORE_BF16 ? 4 : 8;
  void* dst = c->ws + c->lay.ckpt + elem * (size_t)slot * c->cfg.max_batch * (size_t)c->N;
  cudaError_t e = launch_ckpt_copy(true, reinterpret_cast<const float2*>(psi), nullptr, dst,
                                   c->cfg.storage == QML_STORE_BF16 ? 1 : 0, (long long)B * c->N,
                                   static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return QML_ERR_CUDA;
  c->ckpt_batch[slot] = B;
  return QML_OK;
}

qml_status qml_ckpt_restore(qml_ctx* c, int slot, float* psi, int B, void* stream) {
  qml_status st = ckpt_common(c, slot, psi, B);
  if (st != QML_OK) return st;
  if (c->ckpt_batch[slot] != B) return QML_ERR_CKPT_MISMATCH;
  DeviceGuard g(c->device);
  if (int8_slots(c))
    return cuda_status(copy_slot8(c, false, slot, reinterpret_cast<float2*>(psi), B, static_cast<cudaStream_t>(stream)));
  const size_t elem = c->cfg.storage == QML_STORE_BF16 ? 4 : 8;
  void* src = c->ws + c->lay.ckpt + elem * (size_t)slot * c->cfg.max_batch * (size_t)c->N;
  return cuda_status(launch_ckpt_copy(false, nullptr, reinterpret_cast<float2*>(psi), src,
                                      c->cfg.storage == QML_STORE_BF16 ? 1 : 0, (long long)B * c->N,
                                      static_cast<cudaStream_t>(stream)));
}

qml_status qml_expect_z0(qml_ctx* c, const float* psi, int B, float* expect, void* stream) {
  qml_status st = check_ready(c, B);
  if (st != QML_OK) return st;
  if (!psi || !expect || misaligned(psi, 8)) return QML_ERR_INVALID_ARG;
  DeviceGuard g(c->device);
  return cuda_status(launch_expect(reinterpret_cast<const float2*>(psi), B, c->cfg.n_qubits,
                                   at<double>(c, c->lay.exp_partial), expect,
                                   at<unsigned>(c, c->lay.status), static_cast<cudaStream_t>(stream)));
}

qml_status qml_set_observable(qml_ctx* c, int n_terms, const char* paulis, const double* coeffs) {
  if (!c || n_terms < 0 || n_terms > QML_MAX_OBS_TERMS) return QML_ERR_INVALID_ARG;
  ++c->gen;  // a captured host step no longer matches
  if (n_terms > 0 && (!paulis || !coeffs)) return QML_ERR_INVALID_ARG;
  const int n = c->cfg.n_qubits;
  struct Term {
    uint32_t x, z;
    int ny;
    double c;
  };
  std::vector<Term> t((size_t)n_terms);
  for (int k = 0; k < n_terms; ++k) {
    Term& tk = t[(size_t)k];
    tk.x = tk.z = 0;
    tk.ny = 0;
    tk.c = coeffs[k];
    if (!(tk.c == tk.c) || tk.c - tk.c != 0.0) return QML_ERR_INVALID_ARG;  // NaN or infinite
    for (int q = 0; q < n; ++q) {
      const char ch = paulis[(size_t)k * n + q];
      if (ch == 'X' || ch == 'Y') tk.x |= 1u << q;
      if (ch == 'Z' || ch == 'Y') tk.z |= 1u << q;
      if (ch == 'Y') ++tk.ny;
      if (ch != 'I' && ch != 'X' && ch != 'Y' && ch != 'Z') return QML_ERR_INVALID_ARG;
    }
  }
  std::stable_sort(t.begin(), t.end(), [](const Term& a, const Term& b) { return a.x < b.x; });
  c->obs_terms.clear();
  c->obs_groups.clear();
  for (const Term& tk : t) {
    if (c->obs_groups.empty() || c->obs_groups.back().x != tk.x)
      c->obs_groups.push_back({tk.x, (int)c->obs_terms.size(), 0, 0});
    c->obs_groups.back().count++;
    c->obs_terms.push_back({tk.z, tk.ny, tk.c});
  }
  c->obs_dirty = true;
  return QML_OK;
}

// The schedule, its device copies and the workspace layout belong together:
// after a change of schedule the caller sets the workspace again.
static void drop_workspace(qml_ctx* c) {
  c->ws = nullptr;
  c->ws_bytes = 0;
  c->maps.clear();
}

// Back to the schedule of qml_create (CZ entanglers, or CNOT lists through
// the one-layer schedules).
static void restore_default_plan(qml_ctx* c) {
  Plan p;
  make_plan(c->cfg.n_qubits, c->cfg.n_layers, c->cfg.ckpt_block, &p);  // succeeded in qml_create
  c->plan = p;
  flatten_plan(p, &c->dpass);
  flatten_plan(p, &c->dpass_split, true);
  c->undo = undo_order(p, c->dpass_split);
  set_pass_entangler(p, c->bonds, &c->dpass);
  set_pass_entangler(p, c->bonds, &c->dpass_split);
  c->cnot_fused = false;
  if (c->f64) set_f64_tiles(c);
  if (c->ws) drop_workspace(c);
}

qml_status qml_set_entangler(qml_ctx* c, int n_bonds, const int* bonds) {
  if (!c || n_bonds < 0 || n_bonds > QML_MAX_BONDS || (n_bonds > 0 && !bonds)) return QML_ERR_INVALID_ARG;
  ++c->gen;  // a captured host step no longer matches
  const int n = c->cfg.n_qubits;
  Bonds b;
  for (int e = 0; e < n_bonds; ++e) {
    const int x = bonds[2 * e], y = bonds[2 * e + 1];
    if (x < 0 || y < 0 || x >= n || y >= n || x == y) return QML_ERR_INVALID_ARG;
    b.push_back({x, y});
  }
  c->bonds = b;
  set_bond_masks(c);
  if (c->cnot_fused) restore_default_plan(c);
  set_pass_entangler(c->plan, c->bonds, &c->dpass);
  set_pass_entangler(c->plan, c->bonds, &c->dpass_split);
  c->cnot = false;
  c->cnot_pairs.clear();
  return QML_OK;
}

qml_status qml_set_entangler_cnot(qml_ctx* c, int n_pairs, const int* pairs) {
  if (!c || n_pairs < 1 || n_pairs > QML_MAX_BONDS || !pairs) return QML_ERR_INVALID_ARG;
  ++c->gen;  // a captured host step no longer matches
  const int n = c->cfg.n_qubits;
  std::vector<std::pair<int, int>> v;
  for (int e = 0; e < n_pairs; ++e) {
    const int ct = pairs[2 * e], tg = pairs[2 * e + 1];
    if (ct < 0 || tg < 0 || ct >= n || tg >= n || ct == tg) return QML_ERR_INVALID_ARG;
    v.push_back({ct, tg});
  }

  Plan p1;
  if (!make_plan(n, 1, 0, &p1).empty()) return QML_ERR_UNSUPPORTED;
  std::vector<DevPass> d;
  flatten_plan(p1, &d);
  set_pass_entangler(p1, Bonds{}, &d);  // the one-layer passes keep no CZ
  for (int var = 0; var < 4; ++var) {
    c->sub[var] = d;
    const bool encodes = (var & 2) != 0, standard = (var & 1) != 0;
    if (!encodes) c->sub[var][0].gen = 0;  // later layers load the previous layer's state
    if (!standard) c->sub[var].back().last = 0;
  }
  // the layer's CNOT list as a map of index bits: M (in list order) and M^-1,
  // on the working-state addresses (the passes keep the state there; the
  // map in address bits is M with its input and output bits renamed)
  auto to_addr = [&](uint32_t qbits) {
    uint32_t a = 0;
    for (int q = 0; q < n; ++q)
      if ((qbits >> q) & 1u) a |= 1u << p1.addr_of[q];
    return a;
  };
  for (int k = 0; k < kMaxQubits; ++k)
    c->cnot_bwd.col[k] = c->cnot_fwd.col[k] = c->cnot_bwd_q.col[k] = c->cnot_fwd_q.col[k] = 0;
  for (int q = 0; q < n; ++q) {
    uint32_t fwd = 1u << q, inv = 1u << q;
    for (const auto& e : v) fwd ^= ((fwd >> e.first) & 1u) << e.second;
    for (auto it = v.rbegin(); it != v.rend(); ++it) inv ^= ((inv >> it->first) & 1u) << it->second;
    c->cnot_bwd.col[p1.addr_of[q]] = to_addr(fwd);
    c->cnot_fwd.col[p1.addr_of[q]] = to_addr(inv);
    c->cnot_bwd_q.col[q] = fwd;
    c->cnot_fwd_q.col[q] = inv;
  }
  c->sub_mask.clear();
  for (const DevPass& dp : c->sub[0]) c->sub_mask.push_back(f64_tile_mask(dp, n));
  c->plan1 = p1;
  c->cnot_pairs = v;
  c->cnot = true;
  // fused schedule: M1 and M2 of every layer inside the rotation passes
  bool fused = false;
  {
    CnotLayers cl;
    Plan fp;
    if (factor_cnot_layer(n, v, &cl) && make_plan(n, c->cfg.n_layers, c->cfg.ckpt_block, &fp, &cl).empty()) {
      std::vector<DevPass> dp, dps;
      flatten_plan(fp, &dp);
      flatten_plan(fp, &dps, true);
      set_pass_entangler(fp, Bonds{}, &dp);
      set_pass_entangler(fp, Bonds{}, &dps);
      c->plan = fp;
      c->dpass = dp;
      c->dpass_split = dps;
      c->undo = undo_order(fp, dps);
      c->cnot_fused = fused = true;
      c->cnot_map = cl;
    }
  }
  if (!fused && c->cnot_fused) restore_default_plan(c);
  if (c->f64) set_f64_tiles(c);
  if (c->ws) drop_workspace(c);  // the schedule's device copies and the layout change with it
  compute_layout(c);  // the gathers need a second state buffer in the workspace
  return QML_OK;
}

int qml_entangler_kind(const qml_ctx* c) { return c ? (c->cnot ? 1 : 0) : -1; }

int qml_debug_entangler_map(const qml_ctx* c, int* out, int cap) {
  if (!c || !c->cnot) return -1;
  const int n = c->cfg.n_qubits;
  std::vector<int> v;
  v.push_back(n);
  for (int q = 0; q < n; ++q) v.push_back((int)c->cnot_bwd_q.col[q]);  // M
  for (int q = 0; q < n; ++q) v.push_back((int)c->cnot_fwd_q.col[q]);  // M^-1
  for (int a = 0; a < n; ++a) v.push_back((int)c->cnot_bwd.col[a]);    // M on working-state addresses
  for (int a = 0; a < n; ++a) v.push_back((int)c->cnot_fwd.col[a]);
  v.push_back(c->cnot_fused ? 1 : 0);  // then M1 and M2 of the fused schedule (qubit bits)
  for (int g = 0; g < 2; ++g)
    for (int q = 0; q < n; ++q) v.push_back(c->cnot_fused ? (int)c->cnot_map.fwd[g][q] : 0);
  for (int i = 0; i < (int)v.size() && out && i < cap; ++i) out[i] = v[i];
  return (int)v.size();
}

qml_status qml_set_reupload(qml_ctx* c, int on) {
  if (!c) return QML_ERR_INVALID_ARG;
  ++c->gen;  // a captured host step no longer matches
  if (on && c->slow && !c->f64) return QML_ERR_UNSUPPORTED;  // fp32, n < 5: batch-unit register bits
  c->reupload = on != 0;
  return QML_OK;
}

int qml_reupload(const qml_ctx* c) { return c ? (c->reupload ? 1 : 0) : -1; }

int qml_split_form(const qml_ctx* c) { return c ? ((use_split(c) || use_split64(c)) ? 1 : 0) : -1; }

int qml_entangler_bonds(const qml_ctx* c) {
  return c ? (int)(c->cnot ? c->cnot_pairs.size() : c->bonds.size()) : -1;
}

int qml_observable_terms(const qml_ctx* c) { return c ? (int)c->obs_terms.size() : -1; }

qml_status qml_expect_observable(qml_ctx* c, const float* psi, int B, float* expect, void* stream) {
  qml_status st = check_ready(c, B);
  if (st != QML_OK) return st;
  if (!psi || !expect || misaligned(psi, 8)) return QML_ERR_INVALID_ARG;
  DeviceGuard g(c->device);
  return cuda_status(launch_expectation(c, reinterpret_cast<const float2*>(psi), B, expect,
                                        static_cast<cudaStream_t>(stream)));
}

// The copies and launches of one host step, enqueued on s (no synchronisation).
static qml_status enqueue_step_host(qml_ctx* c, const float* x_h, const float* theta_h, const float* y_h, int B,
                                    float* expect_h, float* loss_h, float* grad_h, cudaStream_t s) {
  const int n = c->cfg.n_qubits, L = c->cfg.n_layers;
  const Layout& l = c->lay;
  cudaError_t e = cudaMemcpyAsync(c->ws + l.h_x, x_h, sizeof(float) * (size_t)B * n, cudaMemcpyHostToDevice, s);
  if (e == cudaSuccess)
    e = cudaMemcpyAsync(c->ws + l.h_theta, theta_h, sizeof(float) * (size_t)L * n * 3, cudaMemcpyHostToDevice, s);
  if (e == cudaSuccess) e = cudaMemcpyAsync(c->ws + l.h_y, y_h, sizeof(float) * (size_t)B, cudaMemcpyHostToDevice, s);
  if (e != cudaSuccess) return QML_ERR_CUDA;
  float2* psi = at<float2>(c, l.h_psi);
  float2* lam = at<float2>(c, l.h_lam);
  qml_status st = run_forward(c, at<float>(c, l.h_theta), at<float>(c, l.h_x), B, psi, at<float>(c, l.h_E), s);
  if (st != QML_OK) return st;
  e = launch_loss_seed(at<float>(c, l.h_E), at<float>(c, l.h_y), B, at<float>(c, l.h_g), at<float>(c, l.h_loss), s);
  ++c->launches;
  if (e != cudaSuccess) return QML_ERR_CUDA;
  st = run_backward(c, at<float>(c, l.h_theta), at<float>(c, l.h_x), B, psi, lam, at<float>(c, l.h_g),
                    at<float>(c, l.h_grad), s);
  if (st != QML_OK) return st;
  e = cudaMemcpyAsync(grad_h, c->ws + l.h_grad, sizeof(float) * (size_t)L * n * 3, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess && expect_h)
    e = cudaMemcpyAsync(expect_h, c->ws + l.h_E, sizeof(float) * (size_t)B, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess && loss_h) e = cudaMemcpyAsync(loss_h, c->ws + l.h_loss, sizeof(float), cudaMemcpyDeviceToHost, s);
  return cuda_status(e);
}

static void drop_host_graph(qml_ctx* c) {
  if (c->hg.exec) cudaGraphExecDestroy(c->hg.exec);
  c->hg = qml_ctx::HostGraph{};
}

// Capture one host step on the context's own stream into an executable graph
// (false, and nothing kept, if any part of it cannot be captured).
static bool capture_step_host(qml_ctx* c, const float* x_h, const float* theta_h, const float* y_h, int B,
                              float* expect_h, float* loss_h, float* grad_h) {
  if (!c->cap && cudaStreamCreateWithFlags(&c->cap, cudaStreamNonBlocking) != cudaSuccess) {
    cudaGetLastError();
    c->cap = nullptr;
    return false;
  }
  const long long l0 = c->launches;
  if (cudaStreamBeginCapture(c->cap, cudaStreamCaptureModeThreadLocal) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  const qml_status st = enqueue_step_host(c, x_h, theta_h, y_h, B, expect_h, loss_h, grad_h, c->cap);
  cudaGraph_t g = nullptr;
  const cudaError_t e = cudaStreamEndCapture(c->cap, &g);
  const long long nl = c->launches - l0;
  c->launches = l0;
  bool ok = st == QML_OK && e == cudaSuccess && g != nullptr;
  cudaGraphExec_t exec = nullptr;
  if (ok) ok = cudaGraphInstantiate(&exec, g, 0) == cudaSuccess;
  if (g) cudaGraphDestroy(g);
  if (!ok) {
    cudaGetLastError();
    if (exec) cudaGraphExecDestroy(exec);
    return false;
  }
  c->hg.exec = exec;
  c->hg.launches = nl;
  return true;
}

qml_status qml_step_host(qml_ctx* c, const float* x_h, const float* theta_h, const float* y_h, int B,
                         float* expect_h, float* loss_h, float* grad_h, void* stream) {
  qml_status st = check_ready(c, B);
  if (st != QML_OK) return st;
  if (!x_h || !theta_h || !y_h || !grad_h) return QML_ERR_INVALID_ARG;
  if (c->ws_bytes < c->lay.host_total) return QML_ERR_WORKSPACE;
  DeviceGuard g(c->device);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const void* key[7] = {x_h, theta_h, y_h, expect_h, loss_h, grad_h, c->ws};
  qml_ctx::HostGraph& hg = c->hg;
  const bool same = hg.B == B && hg.gen == c->gen && std::memcmp(hg.key, key, sizeof(key)) == 0;
  if (!same) {
    drop_host_graph(c);
    std::memcpy(hg.key, key, sizeof(key));
    hg.B = B;
    hg.gen = c->gen;
  }
  // the same call again (timing off, every upload done by the eager run):
  // capture it once, then replay
  if (same && hg.seen && !hg.exec && !hg.failed && !c->timing)
    hg.failed = !capture_step_host(c, x_h, theta_h, y_h, B, expect_h, loss_h, grad_h);
  cudaError_t e;
  if (same && hg.exec && !c->timing) {
    e = cudaGraphLaunch(hg.exec, s);
    c->launches += hg.launches;
  } else {
    st = enqueue_step_host(c, x_h, theta_h, y_h, B, expect_h, loss_h, grad_h, s);
    if (st != QML_OK) return st;
    hg.seen = true;
    e = cudaSuccess;
  }
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  return cuda_status(e);
}

qml_status qml_sync(qml_ctx* c, void* stream) {
  if (!c) return QML_ERR_INVALID_ARG;
  if (!c->ws) return QML_ERR_WORKSPACE;
  DeviceGuard g(c->device);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  unsigned word = 0;
  cudaError_t e = cudaMemcpyAsync(&word, c->ws + c->lay.status, sizeof(word), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess) e = cudaMemsetAsync(c->ws + c->lay.status, 0, sizeof(word), s);
  if (e != cudaSuccess) return QML_ERR_CUDA;
  for (int code = 1; code < 32; ++code)
    if (word & (1u << code)) return static_cast<qml_status>(code);
  return QML_OK;
}

qml_status qml_enable_timing(qml_ctx* c, int enable) {
  if (!c) return QML_ERR_INVALID_ARG;
  c->timing = enable != 0;
  return QML_OK;
}

qml_status qml_read_timing(qml_ctx* c, double* fwd_ms, long long* fwd_n, double* bwd_ms, long long* bwd_n) {
  if (!c) return QML_ERR_INVALID_ARG;
  DeviceGuard g(c->device);
  double f = 0.0, b = 0.0;
  long long nf = 0, nb = 0;
  qml_status st = QML_OK;
  for (auto& sp : c->spans) {
    float ms = 0.f;
    if (cudaEventSynchronize(sp.b) != cudaSuccess || cudaEventElapsedTime(&ms, sp.a, sp.b) != cudaSuccess) st = QML_ERR_CUDA;
    if (sp.bwd) { b += ms; nb += sp.passes; } else { f += ms; nf += sp.passes; }
    c->spare.push_back(sp.a);
    c->spare.push_back(sp.b);
  }
  c->spans.clear();
  if (fwd_ms) *fwd_ms = f;
  if (fwd_n) *fwd_n = nf;
  if (bwd_ms) *bwd_ms = b;
  if (bwd_n) *bwd_n = nb;
  return st;
}

long long qml_launch_count(const qml_ctx* c) { return c ? c->launches : -1; }

int qml_debug_schedule(const qml_ctx* c, int* out, int cap) {
  if (!c) return -1;
  std::vector<int> v = describe_plan(c->plan);
  if (out)
    for (int i = 0; i < cap && i < (int)v.size(); ++i) out[i] = v[i];
  return (int)v.size();
}

int qml_debug_layouts(int* out, int cap) { return debug_layouts(out, out ? cap : 0); }

int qml_debug_tile_view(const qml_ctx* c, int pass, int* out, int cap) {
  if (!c || pass < 0 || pass >= (int)c->dpass.size()) return -1;
  const DevPass& d = c->dpass[pass];
  std::vector<int> v;
  v.push_back(d.tma);
  for (int i = 0; i < kTmaRank; ++i) {
    v.push_back(d.tma_kind[i]);
    v.push_back(d.tma_qlo[i]);
    v.push_back(d.tma_bits[i]);
    v.push_back(d.tma_shift[i]);
  }
  for (int b = 0; b < kTileBits; ++b) {
    v.push_back(d.tile_q[b]);
    v.push_back(d.sstride[b]);
  }
  v.push_back(d.n_out);
  for (int i = 0; i < d.n_out; ++i) v.push_back(d.out_q[i]);
  for (int b = 0; b < kTileBits; ++b) v.push_back(d.tile_abit[b] ? __builtin_ctz(d.tile_abit[b]) : -1);
  for (int i = 0; i < d.n_out; ++i) v.push_back(__builtin_ctz(d.out_abit[i]));
  v.push_back(d.variant);
  if (out)
    for (int i = 0; i < cap && i < (int)v.size(); ++i) out[i] = v[i];
  return (int)v.size();
}


// ------------------------------------------------------------ fp64 mode

qml_status qml_forward_expect_f64(qml_ctx* c, const double* theta, const double* x, int B, double* psi,
                                  double* expect, void* stream) {
  qml_status st = check_ready(c, B, true);
  if (st != QML_OK) return st;
  if (!theta || !x || !psi || !expect || misaligned(psi, 16)) return QML_ERR_INVALID_ARG;
  DeviceGuard g(c->device);
  if (c->fault == qml_ctx::FAULT_NAN) {  // injected: the first angle becomes NaN (in a copy of theta)
    double* t = at<double>(c, c->lay.fault_theta);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const size_t bytes = sizeof(double) * 3 * (size_t)c->cfg.n_layers * c->cfg.n_qubits;
    cudaError_t e = cudaMemcpyAsync(t, theta, bytes, cudaMemcpyDeviceToDevice, s);
    if (e == cudaSuccess) e = cudaMemsetAsync(t, 0xff, sizeof(double), s);
    if (e != cudaSuccess) return QML_ERR_CUDA;
    theta = t;
  }
  return run_forward64(c, theta, x, B, reinterpret_cast<double2*>(psi), expect, static_cast<cudaStream_t>(stream));
}

qml_status qml_backward_adjoint_f64(qml_ctx* c, const double* theta, const double* x, int B, double* psi,
                                    double* lambda, const double* dLdE, double* grad, void* stream) {
  qml_status st = check_ready(c, B, true);
  if (st != QML_OK) return st;
  if (!theta || !psi || !lambda || !dLdE || !grad || misaligned(psi, 16) || misaligned(lambda, 16))
    return QML_ERR_INVALID_ARG;
  if (psi == lambda) return QML_ERR_INVALID_ARG;
  if (c->reupload && !x) return QML_ERR_INVALID_ARG;
  DeviceGuard g(c->device);
  return run_backward64(c, theta, x, B, reinterpret_cast<double2*>(psi), reinterpret_cast<double2*>(lambda),
                        dLdE, grad, static_cast<cudaStream_t>(stream));
}

qml_status qml_loss_seed_f64(qml_ctx* c, const double* expect, const double* y, int B, double* g_out,
                             double* loss, void* stream) {
  qml_status st = check_ready(c, B, true);
  if (st != QML_OK) return st;
  if (!expect || !y) return QML_ERR_INVALID_ARG;
  DeviceGuard g(c->device);
  ++c->launches;
  return cuda_status(launch_loss_seed64(expect, y, B, g_out, loss, static_cast<cudaStream_t>(stream)));
}

qml_status qml_step_host_f64(qml_ctx* c, const double* x_h, const double* theta_h, const double* y_h, int B,
                             double* expect_h, double* loss_h, double* grad_h, void* stream) {
  qml_status st = check_ready(c, B, true);
  if (st != QML_OK) return st;
  if (!x_h || !theta_h || !y_h || !grad_h) return QML_ERR_INVALID_ARG;
  if (c->ws_bytes < c->lay.host_total) return QML_ERR_WORKSPACE;
  DeviceGuard g(c->device);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int n = c->cfg.n_qubits, L = c->cfg.n_layers;
  const Layout& l = c->lay;
  const size_t P = (size_t)L * n * 3;
  cudaError_t e = cudaMemcpyAsync(c->ws + l.h_x, x_h, sizeof(double) * (size_t)B * n, cudaMemcpyHostToDevice, s);
  if (e == cudaSuccess) e = cudaMemcpyAsync(c->ws + l.h_theta, theta_h, sizeof(double) * P, cudaMemcpyHostToDevice, s);
  if (e == cudaSuccess) e = cudaMemcpyAsync(c->ws + l.h_y, y_h, sizeof(double) * (size_t)B, cudaMemcpyHostToDevice, s);
  if (e != cudaSuccess) return QML_ERR_CUDA;
  double* x = at<double>(c, l.h_x);
  double* th = at<double>(c, l.h_theta);
  double2* psi = at<double2>(c, l.h_psi);
  double2* lam = at<double2>(c, l.h_lam);
  double* E = at<double>(c, l.h_E);
  double* gv = at<double>(c, l.h_g);
  double* loss = at<double>(c, l.h_loss);
  double* grad = at<double>(c, l.h_grad);
  st = run_forward64(c, th, x, B, psi, E, s);
  if (st != QML_OK) return st;
  ++c->launches;
  if (launch_loss_seed64(E, at<double>(c, l.h_y), B, gv, loss, s) != cudaSuccess) return QML_ERR_CUDA;
  st = run_backward64(c, th, x, B, psi, lam, gv, grad, s);
  if (st != QML_OK) return st;
  e = cudaMemcpyAsync(grad_h, grad, sizeof(double) * P, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess && expect_h)
    e = cudaMemcpyAsync(expect_h, E, sizeof(double) * (size_t)B, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess && loss_h) e = cudaMemcpyAsync(loss_h, loss, sizeof(double), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  return cuda_status(e);
}

}  // extern "C"
