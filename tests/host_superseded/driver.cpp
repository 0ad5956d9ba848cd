// Every call on a static handle that a later one on its GPU has superseded is
// refused, settings included, and leaves the later one as it was.  On the
// stand-ins of the handle's checks; prints "ok".
#define main handle_main
#include "../host_handle/driver.cpp"
#undef main

namespace muon {
hipError_t launch_mx4_quantize(const Mx4List&, bool, bool, RoundingSeed, hipStream_t) { return g_launch; }
hipError_t launch_precond_refresh_mx4(const PrecondBlockDev&, const Mx4Acts&, float, uint32_t*, hipStream_t) { return g_launch; }
hipError_t launch_precond_accumulate_mx4(const PrecondBlockDev&, const Mx4Acts&, double, uint32_t*, hipStream_t) {
  return g_launch;
}
}  // namespace muon

int main() {
  Request r;
  r.tensors.erase(r.tensors.begin() + 1, r.tensors.begin() + 8);     // what fits the array
  const auto init = [&](muon_handle_t* h) {
    return muon_init_static(h, r.tensors.data(), int32_t(r.tensors.size()), &r.slot, 1, &r.hp, nullptr);
  };
  const muon_tensor_t& t = r.tensors[0];
  uint8_t* const c = reinterpret_cast<uint8_t*>(uintptr_t(1) << 45);
  uint8_t* const e = reinterpret_cast<uint8_t*>(uintptr_t(1) << 46);
  muon_mx4_t w;
  std::memset(&w, 0, sizeof(w));
  w.values = t.param;
  w.rows = t.rows, w.cols = t.cols, w.ld = t.ld_param, w.dtype = t.dtype;
  w.row_codes = c, w.row_scales = e;
  w.ld_row_codes = (t.cols + 31) / 32 * 16, w.ld_row_scales = (t.cols + 127) / 128 * 4;
  float ms[512];
  int32_t n = 0;
  int64_t steps = 0;
  uint32_t flags = 0;
  muon_handle_t h = nullptr, later = nullptr;
  const struct { const char* name; std::function<muon_status_t()> call; } calls[] = {
      {"step", [&] { return muon_step(h, -1.f, nullptr); }},
      {"step_timed", [&] { return muon_step_timed(h, -1.f, nullptr, ms, 512, &n); }},
      {"set_adam_step", [&] { return muon_set_adam_step(h, 3, nullptr); }},
      {"get_adam_step", [&] { return muon_get_adam_step(h, nullptr, &steps); }},
      {"set_rounding_seed", [&] { return muon_set_rounding_seed(h, 7); }},
      {"set_max_grad_norm", [&] { return muon_set_max_grad_norm(h, 0.f, nullptr); }},
      {"set_mx4_weights", [&] { return muon_set_mx4_weights(h, &w, 1); }},
      {"set_mx4_weights, off", [&] { return muon_set_mx4_weights(h, nullptr, 0); }},
      {"accumulate", [&] { return muon_precond_accumulate(h, 0, 0, c, 8, 768, MUON_BF16, 0.5f, nullptr); }},
      {"accumulate_mx4", [&] { return muon_precond_accumulate_mx4(h, 0, 0, c, e, 64, 32, 4, 0.5, nullptr); }},
      {"refresh_mx4", [&] { return muon_precond_refresh_mx4(h, 0, 0, c, e, 64, 32, 4, 0.5f, nullptr); }},
      {"refresh_accumulated", [&] { return muon_precond_refresh_accumulated(h, 0, 0, 0.5f, 1, nullptr); }},
      {"sums", [&] { return muon_precond_sums(h, 0, 0, nullptr, nullptr, nullptr); }},
      {"get_flags", [&] { return muon_get_flags(h, nullptr, 0, &flags); }},
  };
  CHECK(init(&h) == MUON_OK, "init: %s", muon_last_error());
  for (const auto& x : calls) CHECK(x.call() == MUON_OK, "%s, before: %s", x.name, muon_last_error());
  CHECK(init(&later) == MUON_OK, "init: %s", muon_last_error());
  for (const auto& x : calls) CHECK(x.call() == MUON_ERR_BAD_ARG, "%s is not refused", x.name);
  (void)muon_destroy(h);
  h = later;
  for (const auto& x : calls) CHECK(x.call() == MUON_OK, "%s, of the later one: %s", x.name, muon_last_error());
  (void)muon_destroy(later);
  if (!g_bad) std::printf("ok\n");
  return g_bad ? 1 : 0;
}
