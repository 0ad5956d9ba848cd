// The handle's host code without a GPU: the HIP runtime calls and the kernel
// launchers it makes are stand-ins that count what lives, and operator new can
// be told to fail.  argv[1] names the check; each prints "ok" at the end.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <functional>
#include <new>
#include <string>
#include <vector>

#include <hip/hip_runtime.h>

#include "muon.h"
#include "muon_internal.h"

// ------------------------------------------------------------- stand-ins

static long g_live = 0, g_fail_at = 0, g_news = 0;      // allocations; 0: none fails
static long g_streams = 0, g_events = 0, g_objects = 0, g_fail_object = 0;
static hipError_t g_launch = hipSuccess, g_sync = hipSuccess;

void* operator new(size_t n) {
  ++g_news;
  if (g_fail_at && --g_fail_at == 0) throw std::bad_alloc();
  void* p = std::malloc(n ? n : 1);
  if (!p) throw std::bad_alloc();
  ++g_live;
  return p;
}
void operator delete(void* p) noexcept {
  if (p) --g_live;
  std::free(p);
}
void operator delete(void* p, size_t) noexcept { operator delete(p); }

template <typename T>
static hipError_t make(T* out, long& live) {
  if (g_fail_object && --g_fail_object == 0) return hipErrorOutOfMemory;
  ++live;
  *out = reinterpret_cast<T>(++g_objects);
  return hipSuccess;
}

extern "C" {
hipError_t hipMemsetAsync(void*, int, size_t, hipStream_t) { return hipSuccess; }
hipError_t hipMemcpyAsync(void*, const void*, size_t, hipMemcpyKind, hipStream_t) { return hipSuccess; }
hipError_t hipMemcpy(void* dst, const void*, size_t n, hipMemcpyKind) {
  std::memset(dst, 0, n);
  return hipSuccess;
}
hipError_t hipStreamSynchronize(hipStream_t) { return g_sync; }
hipError_t hipStreamCreateWithFlags(hipStream_t* s, unsigned int) { return make(s, g_streams); }
hipError_t hipStreamDestroy(hipStream_t) { return --g_streams, hipSuccess; }
hipError_t hipEventCreateWithFlags(hipEvent_t* e, unsigned int) { return make(e, g_events); }
hipError_t hipEventCreate(hipEvent_t* e) { return make(e, g_events); }
hipError_t hipEventDestroy(hipEvent_t) { return --g_events, hipSuccess; }
hipError_t hipEventRecord(hipEvent_t, hipStream_t) { return hipSuccess; }
hipError_t hipEventSynchronize(hipEvent_t) { return hipSuccess; }
hipError_t hipEventElapsedTime(float* ms, hipEvent_t, hipEvent_t) { return *ms = 1.f, hipSuccess; }
hipError_t hipStreamWaitEvent(hipStream_t, hipEvent_t, unsigned int) { return hipSuccess; }
hipError_t hipGetDevice(int* d) { return *d = 0, hipSuccess; }
hipError_t hipGetSymbolAddress(void** p, const void*) {
  *p = reinterpret_cast<void*>(uintptr_t(1) << 40);
  return hipSuccess;
}
const char* hipGetErrorString(hipError_t) { return "stand-in"; }
int roctxRangePushA(const char*) { return 0; }
int roctxRangePop() { return 0; }
}

namespace muon {
hipError_t launch_momentum(bool, const UnitDev*, const EwTask*, int, const K1Params&, hipStream_t) { return g_launch; }
hipError_t launch_gemm(int, bool, int, const UnitDev*, const GemmTask*, int, const GemmParams&, hipStream_t) {
  return g_launch;
}
hipError_t launch_update(bool, const UnitDev*, const EwTask*, int, const K5Params&, hipStream_t) { return g_launch; }
hipError_t launch_precond_refresh(const PrecondBlockDev&, const void*, int64_t, int64_t, bool, float, uint32_t*,
                                  hipStream_t) {
  return g_launch;
}
hipError_t launch_precond_accumulate(const PrecondBlockDev&, const void*, int64_t, int64_t, bool, float, hipStream_t) {
  return g_launch;
}
hipError_t launch_precond_refresh_accumulated(const PrecondBlockDev&, float, bool, uint32_t*, hipStream_t) {
  return g_launch;
}
hipError_t launch_precond_apply(const PrecondDev*, const ApplyTask*, int, int, hipStream_t) { return g_launch; }
hipError_t launch_identity(uint16_t*, int, int, hipStream_t) { return hipSuccess; }
hipError_t launch_adam_tick(AdamState*, float, float, hipStream_t) { return g_launch; }
hipError_t launch_adam_set(AdamState*, uint32_t, hipStream_t) { return g_launch; }
hipError_t launch_adamw(const AdamDev*, const AdamTask*, int, const AdamParams&, hipStream_t) { return g_launch; }
hipError_t launch_adamw_packed(const PackedDev*, const PackedTask*, const int*, bool, PackedParams, hipStream_t) {
  return g_launch;
}
hipError_t launch_pack_moments(const PackedDev*, const PackedTask*, int, const void*, int64_t, bool, uint32_t*,
                               hipStream_t) {
  return g_launch;
}
hipError_t launch_unpack_moments(const PackedDev*, const PackedTask*, int, void*, int64_t, bool, uint32_t*,
                                 hipStream_t) {
  return g_launch;
}
hipError_t launch_grad_norm(const NormParams&, hipStream_t) { return g_launch; }
}  // namespace muon

// ----------------------------------------------------------------- checks

static int g_bad = 0;
#define CHECK(c, ...)                       \
  do {                                      \
    if (!(c)) {                             \
      std::printf("line %d: ", __LINE__);   \
      std::printf(__VA_ARGS__);             \
      std::printf("\n");                    \
      ++g_bad;                              \
    }                                       \
  } while (0)

// Two lanes of matrices, one with a preconditioner, AdamW of both kinds of moments.
struct Request {
  std::vector<muon_tensor_t> tensors;
  muon_precond_t slot{768, 1, 0};
  muon_hparams_t hp;
  uintptr_t at = uintptr_t(1) << 36;

  uintptr_t take(size_t bytes) {
    const uintptr_t p = at;
    at += (bytes + 4095) / 4096 * 4096;
    return p;
  }
  void add(int64_t rows, int64_t cols, int kind, int bits, int precond) {
    muon_tensor_t t;
    std::memset(&t, 0, sizeof(t));
    t.param = reinterpret_cast<void*>(take(rows * cols * 2));
    t.grad = reinterpret_cast<void*>(take(rows * cols * 2));
    t.momentum = reinterpret_cast<float*>(take(rows * cols * 4 + 8192));
    if (kind == MUON_KIND_ADAMW) t.exp_avg_sq = reinterpret_cast<float*>(take(rows * cols * 4 + 8192));
    t.rows = rows;
    t.cols = t.ld_param = t.ld_grad = t.ld_momentum = cols;
    t.dtype = MUON_BF16;
    t.precond = precond;
    t.lr_mult = 1.f;
    t.kind = kind;
    t.state_bits = bits;
    tensors.push_back(t);
  }
  Request() {
    muon_default_hparams(&hp);
    for (int k = 0; k < 8; ++k) add(768, 768, MUON_KIND_MUON, 0, k ? -1 : 0);
    add(1, 768, MUON_KIND_ADAMW, 0, -1);
    add(300, 64, MUON_KIND_ADAMW, 8, -1);
  }
  muon_status_t init(muon_handle_t* h) {
    size_t bytes = 0;
    const muon_status_t st = muon_workspace_size(tensors.data(), int32_t(tensors.size()), &slot, 1, &hp, &bytes);
    return st != MUON_OK ? st
                         : muon_init(h, tensors.data(), int32_t(tensors.size()), &slot, 1, &hp,
                                     reinterpret_cast<void*>(uintptr_t(1) << 40), bytes, nullptr);
  }
};

// A message longer than any that follows, so that later ones need no room of their own.
static void long_message() {
  Request r;
  r.tensors[9].momentum = r.tensors[8].momentum;
  muon_handle_t h;
  (void)r.init(&h);
}

// Every allocation of muon_init fails in turn, and every stream or event: nothing may stay behind.
static void check_init() {
  Request r;
  long_message();
  muon_handle_t h = nullptr;
  long n = g_news;
  CHECK(r.init(&h) == MUON_OK, "init: %s", muon_last_error());
  n = g_news - n;
  CHECK(g_streams >= 2 && g_events >= 3, "no lanes: %ld streams, %ld events", g_streams, g_events);
  CHECK(muon_destroy(h) == MUON_OK && g_streams == 0 && g_events == 0, "destroy leaves %ld, %ld", g_streams, g_events);
  const long live = g_live;
  for (long k = 1; k <= n; ++k) {
    g_fail_at = k;
    h = nullptr;
    muon_status_t st = MUON_OK;
    try {
      st = r.init(&h);
    } catch (...) {
      CHECK(false, "allocation %ld: an exception left the call", k);
    }
    g_fail_at = 0;
    // a sort that gets no room for its copy does without
    CHECK(st == MUON_ERR_UNSUPPORTED ? !h : st == MUON_OK, "allocation %ld: status %d", k, int(st));
    if (st == MUON_OK) (void)muon_destroy(h);
    CHECK(g_live == live, "allocation %ld: %ld allocations stay behind", k, g_live - live);
    CHECK(g_streams == 0 && g_events == 0, "allocation %ld: %ld streams, %ld events stay behind", k, g_streams, g_events);
    g_live = live;
    g_streams = g_events = 0;
    if (g_bad > 8) return;
  }
  CHECK(r.init(&h) == MUON_OK, "init: %s", muon_last_error());
  const long made = g_streams + g_events;
  (void)muon_destroy(h);
  for (long k = 1; k <= made; ++k) {
    g_fail_object = k;
    CHECK(r.init(&h) == MUON_ERR_HIP && !h, "object %ld: no error", k);
    g_fail_object = 0;
    CHECK(g_live == live && g_streams == 0 && g_events == 0, "object %ld: %ld, %ld, %ld stay behind", k, g_live - live,
          g_streams, g_events);
  }
  g_sync = hipErrorUnknown;
  CHECK(r.init(&h) == MUON_ERR_HIP && !h && g_live == live, "failed upload");
  g_sync = hipSuccess;
}

// No entry point lets an exception out, wherever an allocation fails.
static void check_exceptions() {
  Request r;
  muon_handle_t h = nullptr;
  if (r.init(&h) != MUON_OK) return (void)++g_bad;
  void* const p = reinterpret_cast<void*>(uintptr_t(1) << 45);
  float ms[512];
  int32_t np = 0;
  int64_t steps = 0;
  uint32_t flags = 0;
  const struct { const char* name; std::function<muon_status_t()> call; hipError_t launch; } calls[] = {
      {"step", [&] { return muon_step(h, -1.f, nullptr); }, hipErrorUnknown},
      {"step, bad lr", [&] { return muon_step(h, HUGE_VALF, nullptr); }, hipSuccess},
      {"step_timed", [&] { return muon_step_timed(h, -1.f, nullptr, ms, 512, &np); }, hipSuccess},
      {"step_timed, failing", [&] { return muon_step_timed(h, -1.f, nullptr, ms, 512, &np); }, hipErrorUnknown},
      {"refresh", [&] { return muon_precond_refresh(h, 0, 0, p, 64, 768, MUON_F32, 1.f, nullptr); }, hipErrorUnknown},
      {"refresh, bad slot", [&] { return muon_precond_refresh(h, 7, 0, p, 64, 768, MUON_F32, 1.f, nullptr); }, hipSuccess},
      {"accumulate", [&] { return muon_precond_accumulate(h, 0, 0, p, 64, 768, MUON_F32, 1.f, nullptr); }, hipErrorUnknown},
      {"refresh_accumulated", [&] { return muon_precond_refresh_accumulated(h, 0, 0, 1.f, 1, nullptr); }, hipErrorUnknown},
      {"set_adam_step", [&] { return muon_set_adam_step(h, 5, nullptr); }, hipErrorUnknown},
      {"set_adam_step, bad", [&] { return muon_set_adam_step(h, -5, nullptr); }, hipSuccess},
      {"get_adam_step, null", [&] { return muon_get_adam_step(h, nullptr, nullptr); }, hipSuccess},
      {"get_adam_step", [&] { return muon_get_adam_step(h, nullptr, &steps); }, hipSuccess},
      {"get_flags", [&] { return muon_get_flags(h, nullptr, 1, &flags); }, hipSuccess},
      {"get_flags, null", [&] { return muon_get_flags(h, nullptr, 1, nullptr); }, hipSuccess},
      {"set_rounding_seed, null", [&] { return muon_set_rounding_seed(nullptr, 1); }, hipSuccess},
      {"set_max_grad_norm", [&] { return muon_set_max_grad_norm(h, 1.f, nullptr); }, hipSuccess},
      {"set_max_grad_norm, alias", [&] { return muon_set_max_grad_norm(h, 1.f, static_cast<float*>(r.tensors[9].param)); }, hipSuccess},
      {"pack", [&] { return muon_pack_moments(h, p, MUON_F32, nullptr); }, hipErrorUnknown},
      {"unpack", [&] { return muon_unpack_moments(h, p, MUON_F32, nullptr); }, hipErrorUnknown},
  };
  for (const auto& c : calls) {
    for (long k = 1; k < 64; ++k) {
      g_launch = c.launch;
      g_sync = c.launch;
      g_fail_at = k;
      try {
        (void)c.call();
      } catch (...) {
        CHECK(false, "%s: an exception left the call at allocation %ld", c.name, k);
      }
      const bool reached = g_fail_at == 0;
      g_fail_at = 0;
      g_launch = g_sync = hipSuccess;
      if (!reached) break;
    }
  }
  // a handle whose last stream fails is freed all the same
  g_sync = hipErrorUnknown;
  g_fail_at = 1;
  try {
    CHECK(muon_destroy(h) != MUON_OK, "destroy");
  } catch (...) {
    CHECK(false, "destroy: an exception left the call");
  }
  g_fail_at = 0;
  g_sync = hipSuccess;
  CHECK(g_streams == 0 && g_events == 0, "destroy leaves %ld streams, %ld events", g_streams, g_events);
}

// Names handed out stay as they are while the norm is switched on and off.
static void check_names() {
  Request r;
  muon_handle_t h = nullptr;
  if (r.init(&h) != MUON_OK) return (void)++g_bad;
  int32_t n = 0, with = 0;
  float ms[512];
  CHECK(muon_step_timed(h, -1.f, nullptr, ms, 512, &n) == MUON_OK && n > 10, "%d phases", n);
  std::vector<const char*> names;
  std::vector<std::string> copies;
  for (int32_t k = 0; k < n; ++k) {
    names.push_back(muon_phase_name(h, k));
    copies.push_back(names.back());
  }
  CHECK(copies[0] == "precond_apply" && copies[1] == "adamw", "%s, %s", copies[0].c_str(), copies[1].c_str());
  for (int round = 0; round < 3; ++round) {
    CHECK(muon_set_max_grad_norm(h, 1.f + round, nullptr) == MUON_OK, "set");
    CHECK(std::string(muon_phase_name(h, 0)) == "grad_norm", "%s", muon_phase_name(h, 0));
    for (int32_t k = 0; k < n; ++k) CHECK(muon_phase_name(h, k + 1) == names[k], "phase %d moved", k);
    CHECK(!*muon_phase_name(h, n + 1) && !*muon_phase_name(h, -1), "names past the end");
    CHECK(muon_step_timed(h, -1.f, nullptr, ms, 512, &with) == MUON_OK && with == n + 1, "%d phases", with);
    if (round == 1) continue;
    CHECK(muon_set_max_grad_norm(h, 0.f, nullptr) == MUON_OK, "set");
    for (int32_t k = 0; k < n; ++k) {
      CHECK(muon_phase_name(h, k) == names[k], "phase %d moved back elsewhere", k);
      if (muon_phase_name(h, k) == names[k]) CHECK(copies[k] == names[k], "phase %d reads %s", k, names[k]);
    }
    CHECK(!*muon_phase_name(h, n), "names past the end");
    CHECK(muon_step_timed(h, -1.f, nullptr, ms, 512, &with) == MUON_OK && with == n, "%d phases", with);
  }
  (void)muon_destroy(h);
}

// A static init that fails before it touches the array leaves the earlier handle as it was.
static void check_static() {
  Request r;
  r.tensors.erase(r.tensors.begin() + 1, r.tensors.begin() + 8);     // what fits the array
  const auto init = [&](muon_handle_t* h) {
    return muon_init_static(h, r.tensors.data(), int32_t(r.tensors.size()), &r.slot, 1, &r.hp, nullptr);
  };
  muon_handle_t first = nullptr, second = nullptr;
  long n = g_news;
  CHECK(init(&first) == MUON_OK, "init: %s", muon_last_error());
  n = g_news - n;
  CHECK(muon_step(first, -1.f, nullptr) == MUON_OK, "step: %s", muon_last_error());
  const void* const grad = r.tensors[0].grad;
  r.tensors[0].grad = reinterpret_cast<void*>((uintptr_t(1) << 40) + 4096);     // inside the array
  CHECK(init(&second) == MUON_ERR_ALIASING && !second, "aliasing");
  r.tensors[0].grad = grad;
  CHECK(muon_step(first, -1.f, nullptr) == MUON_OK, "after an aliasing init: %s", muon_last_error());
  for (long k = 1; k <= n; ++k) {
    g_fail_at = k;
    const muon_status_t st = init(&second);
    g_fail_at = 0;
    if (st == MUON_OK) {                       // a sort that does without its copy: this one took over
      (void)muon_destroy(first);
      first = second;
      second = nullptr;
    }
    if (muon_step(first, -1.f, nullptr) != MUON_OK) {
      CHECK(false, "allocation %ld: %s", k, muon_last_error());
      (void)muon_destroy(first);
      if (init(&first) != MUON_OK) return;
    }
  }
  CHECK(init(&second) == MUON_OK, "init: %s", muon_last_error());
  CHECK(muon_step(first, -1.f, nullptr) == MUON_ERR_BAD_ARG, "a superseded handle steps");
  CHECK(muon_step(second, -1.f, nullptr) == MUON_OK, "step: %s", muon_last_error());
  (void)muon_destroy(first);
  (void)muon_destroy(second);
}

int main(int argc, char** argv) {
  const std::string what = argc > 1 ? argv[1] : "";
  if (what == "init") check_init();
  else if (what == "exceptions") check_exceptions();
  else if (what == "names") check_names();
  else if (what == "static") check_static();
  else return 2;
  if (!g_bad) std::printf("ok\n");
  return g_bad ? 1 : 0;
}
