// The host code of microscaled 4-bit floats without a GPU, on the stand-ins and
// the request of the handle's checks: what the launches get, and every
// allocation failing in turn.  argv[1] names the check; each prints "ok".
#define main handle_main
#include "../host_handle/driver.cpp"
#undef main

static std::vector<muon::Mx4List> g_lists;           // of every launch
static std::vector<int> g_what;                      // 0 rounded, 1 + axis read back; 4 added where streamed
static std::vector<muon::Mx4Acts> g_acts;
static int g_record = 1;

namespace muon {
static void record(const Mx4List& l, int what) {
  if (!g_record) return;
  g_lists.push_back(l);
  g_what.push_back(what);
}
hipError_t launch_mx4_quantize(const Mx4List& l, bool, bool, RoundingSeed, hipStream_t) { return record(l, 0), g_launch; }
hipError_t launch_mx4_dequantize(const Mx4List& l, bool, int axis, bool stream, hipStream_t) {
  return record(l, 1 + axis + (stream ? 4 : 0)), g_launch;
}
hipError_t launch_precond_refresh_mx4(const PrecondBlockDev&, const Mx4Acts& a, float, uint32_t*, hipStream_t) {
  if (g_record) g_acts.push_back(a);
  return g_launch;
}
hipError_t launch_precond_accumulate_mx4(const PrecondBlockDev&, const Mx4Acts& a, double, uint32_t*, hipStream_t) {
  if (g_record) g_acts.push_back(a);
  return g_launch;
}
}  // namespace muon

// The k-th matrix of a list, its buffers apart from the others' and from the request's.
static muon_mx4_t matrix(int k, int64_t rows, int64_t cols, int32_t dtype, bool row, bool col) {
  muon_mx4_t x;
  std::memset(&x, 0, sizeof(x));
  const uintptr_t at = (uintptr_t(1) << 44) + uintptr_t(k) * (uintptr_t(1) << 32);
  x.values = reinterpret_cast<void*>(at);
  x.rows = rows;
  x.cols = x.ld = cols;
  x.dtype = dtype;
  auto lines = [](uintptr_t p, int64_t length, uint8_t** codes, uint8_t** scales, int64_t* lc, int64_t* ls) {
    *codes = reinterpret_cast<uint8_t*>(p);
    *scales = reinterpret_cast<uint8_t*>(p + (uintptr_t(1) << 28));
    *lc = (length + 31) / 32 * 16;
    *ls = ((length + 31) / 32 + 3) / 4 * 4;
  };
  if (row) lines(at + (uintptr_t(1) << 30), cols, &x.row_codes, &x.row_scales, &x.ld_row_codes, &x.ld_row_scales);
  if (col) lines(at + (uintptr_t(2) << 30), rows, &x.col_codes, &x.col_scales, &x.ld_col_codes, &x.ld_col_scales);
  return x;
}

// Every matrix is in one launch, in order, with its place, its tiles behind those before it, and launches hold
// one kind each.
static void check_launches() {
  std::vector<muon_mx4_t> list;
  for (int k = 0; k < 300; ++k)
    list.push_back(matrix(k, 1 + 37 * k % 900, 1 + 91 * k % 700, k % 3 ? MUON_BF16 : MUON_F32, k % 5 != 1, k % 5 != 2));
  CHECK(muon_mx4_quantize(list.data(), 300, MUON_ROUND_RANDOM, 1, nullptr) == MUON_OK, "%s", muon_last_error());
  std::vector<int> seen(300, 0);
  for (const muon::Mx4List& l : g_lists) {
    int64_t tiles = 0;
    CHECK(l.n >= 1 && l.n <= muon::kMx4Most, "%d matrices", l.n);
    for (int i = 0; i < l.n; ++i) {
      const muon::Mx4Dev& m = l.m[i];
      const muon_mx4_t& x = list[m.index];
      ++seen[m.index];
      CHECK(i == 0 || l.m[i - 1].index < m.index, "order");
      CHECK(l.tile0[i] == tiles, "matrix %u starts at tile %d of %ld", m.index, l.tile0[i], long(tiles));
      tiles += (x.rows + 127) / 128 * ((x.cols + 127) / 128);
      CHECK(m.tiles_c == (x.cols + 127) / 128 && m.rows == x.rows && m.cols == x.cols && m.ld == x.ld, "sizes");
      CHECK(m.values == x.values && m.row.codes == x.row_codes && m.row.scales == x.row_scales &&
                m.col.codes == x.col_codes && m.col.scales == x.col_scales, "addresses");
      CHECK(int64_t(m.row_ld16) * 16 == x.ld_row_codes && int64_t(m.row_ld4) * 4 == x.ld_row_scales &&
                int64_t(m.col_ld16) * 16 == x.ld_col_codes && int64_t(m.col_ld4) * 4 == x.ld_col_scales, "leading dimensions");
      const muon_mx4_t& first = list[l.m[0].index];
      CHECK(x.dtype == first.dtype && !x.row_codes == !first.row_codes && !x.col_codes == !first.col_codes, "kinds mixed");
    }
    CHECK(l.tiles == tiles, "%d tiles of %ld", l.tiles, long(tiles));
    for (int i = l.n; i < muon::kMx4Most; ++i) CHECK(l.tile0[i] == INT32_MAX, "behind the last");
  }
  for (int k = 0; k < 300; ++k) CHECK(seen[k] == 1, "matrix %d in %d launches", k, seen[k]);
  // leading dimensions whose span passes the end of all addresses
  const auto refused = [](int64_t rows, int64_t ld, int64_t ld_codes, int64_t ld_scales, const char* why) {
    muon_mx4_t x = matrix(0, rows, 32, MUON_F32, true, false);
    x.ld = ld, x.ld_row_codes = ld_codes, x.ld_row_scales = ld_scales;
    for (auto call : {+[](const muon_mx4_t* m) { return muon_mx4_quantize(m, 1, 0, 0, nullptr); },
                      +[](const muon_mx4_t* m) { return muon_mx4_dequantize(m, 1, 1, nullptr); }})
      CHECK(call(&x) == MUON_ERR_BAD_SHAPE && std::string(muon_last_error()).find(why) != std::string::npos, "%s: %s", why,
            muon_last_error());
  };
  refused(1 << 30, 32, int64_t(1) << 35, 4, "along the rows: leading dimensions too large");
  refused(1 << 30, INT64_MAX, 16, 4, "the leading dimension is too large");
  refused(1 << 30, INT64_MAX / 4, 16, 4, "the leading dimension is too large");
  refused(2, INT64_MAX, 16, 4, "the leading dimension is too large");
  // Reading back: streamed where the rows allow it; a small list of both kinds is one launch, a large one two.
  const auto back = [&](std::vector<muon_mx4_t> l, int axis) {
    g_lists.clear(), g_what.clear();
    CHECK(muon_mx4_dequantize(l.data(), int32_t(l.size()), axis, nullptr) == MUON_OK, "%s", muon_last_error());
    return g_what;
  };
  using V = std::vector<int>;
  const muon_mx4_t even = matrix(0, 64, 64, MUON_BF16, true, true), odd = matrix(1, 64, 65, MUON_BF16, true, true);
  const muon_mx4_t large = matrix(2, 8192, 4096, MUON_BF16, true, true), one = matrix(3, 1, 65, MUON_BF16, true, true);
  CHECK(back({even}, 1) == V{6} && back({even, one}, 0) == V{5}, "even rows");
  CHECK(back({odd}, 1) == V{2} && back({even, odd}, 0) == V{1}, "a small list");
  CHECK((back({even, odd, large}, 1) == V{6, 2}), "a large list");
  CHECK(back({}, 1).empty() && muon_mx4_quantize(nullptr, 0, 0, 0, nullptr) == MUON_OK, "no matrices");
}

// The copies of a handle: phases, what its step launches, and a refused list that changes nothing.
static void check_weights() {
  Request r;
  muon_handle_t h = nullptr;
  if (r.init(&h) != MUON_OK) return (void)++g_bad;
  float ms[512];
  int32_t n = 0, with = 0;
  CHECK(muon_step_timed(h, -1.f, nullptr, ms, 512, &n) == MUON_OK, "timed");
  std::vector<muon_mx4_t> list;
  for (int k = 0; k < 10; ++k) {
    const muon_tensor_t& t = r.tensors[k];
    list.push_back(matrix(k, t.rows, t.cols, t.dtype, k != 3, k != 4));
    list.back().values = t.param;
  }
  CHECK(muon_set_mx4_weights(h, list.data(), 10) == MUON_OK, "%s", muon_last_error());
  g_lists.clear();
  CHECK(muon_step(h, -1.f, nullptr) == MUON_OK && g_lists.size() == 3, "%zu launches", g_lists.size());
  CHECK(muon_step_timed(h, -1.f, nullptr, ms, 512, &with) == MUON_OK && with == n + 1, "%d phases", with);
  CHECK(std::string(muon_phase_name(h, n)) == "mx4_weights" && !*muon_phase_name(h, n + 1), "names");
  CHECK(muon_set_max_grad_norm(h, 1.f, nullptr) == MUON_OK, "norm");
  CHECK(std::string(muon_phase_name(h, n + 1)) == "mx4_weights" && std::string(muon_phase_name(h, 0)) == "grad_norm", "names");
  muon_mx4_t bad = list[0];
  bad.rows = 767;
  CHECK(muon_set_mx4_weights(h, &bad, 1) == MUON_ERR_BAD_ARG, "no such param");
  bad = list[0];
  bad.row_codes = static_cast<uint8_t*>(const_cast<void*>(r.tensors[5].grad));
  CHECK(muon_set_mx4_weights(h, &bad, 1) == MUON_ERR_ALIASING, "on a gradient");
  bad.row_codes = reinterpret_cast<uint8_t*>(uintptr_t(1) << 40);
  CHECK(muon_set_mx4_weights(h, &bad, 1) == MUON_ERR_ALIASING, "on the workspace");
  // an allocation that fails leaves the list that was set
  for (long k = 1; k < 32; ++k) {
    g_fail_at = k;
    const muon_status_t st = muon_set_mx4_weights(h, list.data(), 1);
    const bool reached = g_fail_at == 0;
    g_fail_at = 0;
    if (st == MUON_OK) CHECK(muon_set_mx4_weights(h, list.data(), 10) == MUON_OK, "set again");
    else CHECK(st == MUON_ERR_UNSUPPORTED, "allocation %ld: status %d", k, int(st));
    if (!reached) break;
  }
  g_lists.clear();
  CHECK(muon_step(h, -1.f, nullptr) == MUON_OK && g_lists.size() == 3, "%zu launches", g_lists.size());
  CHECK(muon_set_mx4_weights(h, nullptr, 0) == MUON_OK, "off");
  g_lists.clear();
  CHECK(muon_step(h, -1.f, nullptr) == MUON_OK && g_lists.empty(), "still on");
  CHECK(muon_set_mx4_weights(nullptr, nullptr, 0) == MUON_ERR_NULL_ARG, "no handle");
  (void)muon_destroy(h);
}

// Activations: what is refused, what the launch gets, and where the sums are said to lie.
static void check_acts() {
  Request r;
  muon_handle_t h = nullptr;
  if (r.init(&h) != MUON_OK) return (void)++g_bad;
  uint8_t* const c = reinterpret_cast<uint8_t*>(uintptr_t(1) << 45);
  uint8_t* const e = reinterpret_cast<uint8_t*>(uintptr_t(1) << 46);
  const auto both = [&](const uint8_t* pc, const uint8_t* pe, int64_t n, int64_t lc, int64_t le, muon_status_t want) {
    g_acts.clear();
    const muon_status_t a = muon_precond_accumulate_mx4(h, 0, 0, pc, pe, n, lc, le, 0.5, nullptr);
    const muon_status_t b = muon_precond_refresh_mx4(h, 0, 0, pc, pe, n, lc, le, 0.5f, nullptr);
    CHECK(a == want && b == want, "%d and %d for %ld samples, %ld, %ld: %s", int(a), int(b), long(n), long(lc), long(le),
          muon_last_error());
    CHECK(g_acts.size() == (want == MUON_OK ? 2u : 0u), "%zu launches", g_acts.size());
    for (const muon::Mx4Acts& x : g_acts)
      CHECK(x.codes == pc && x.scales == pe && x.n_rows == n && x.ld_codes == lc && x.ld_scales == le, "arguments");
  };
  both(c, e, 1, 16, 4, MUON_OK);
  both(c, e, 33, 32, 4, MUON_OK);
  both(c, e, 4097, 1 << 24, 1 << 24, MUON_OK);
  both(nullptr, e, 1, 16, 4, MUON_ERR_NULL_ARG);
  both(c, nullptr, 1, 16, 4, MUON_ERR_NULL_ARG);
  both(c, e, 0, 16, 4, MUON_ERR_BAD_SHAPE);
  both(c, e, -7, 16, 4, MUON_ERR_BAD_SHAPE);
  both(c, e, 33, 16, 4, MUON_ERR_BAD_SHAPE);
  both(c, e, 129, 80, 4, MUON_ERR_BAD_SHAPE);
  both(c, e, INT64_MAX, 16, 4, MUON_ERR_BAD_SHAPE);
  both(c, e, INT64_MAX, INT64_MAX / 16 * 16, INT64_MAX / 4 * 4, MUON_ERR_UNSUPPORTED);
  both(c + 8, e, 1, 16, 4, MUON_ERR_ALIGNMENT);
  both(c, e + 2, 1, 16, 4, MUON_ERR_ALIGNMENT);
  both(c, e, 1, 24, 4, MUON_ERR_ALIGNMENT);
  both(c, e, 1, 16, 6, MUON_ERR_ALIGNMENT);
  both(c, e, 1, (1 << 24) + 16, 4, MUON_ERR_UNSUPPORTED);
  both(c, e, 1, 16, (1 << 24) + 4, MUON_ERR_UNSUPPORTED);
  for (double beta : {-0.1, 1.1, double(NAN)})
    CHECK(muon_precond_accumulate_mx4(h, 0, 0, c, e, 1, 16, 4, beta, nullptr) == MUON_ERR_BAD_ARG, "beta %g", beta);
  for (float damping : {-0.1f, HUGE_VALF, float(NAN)})
    CHECK(muon_precond_refresh_mx4(h, 0, 0, c, e, 1, 16, 4, damping, nullptr) == MUON_ERR_BAD_ARG, "damping %g", double(damping));
  for (int slot : {-1, 1})
    CHECK(muon_precond_accumulate_mx4(h, slot, 0, c, e, 1, 16, 4, 0.5, nullptr) == MUON_ERR_BAD_ARG &&
              muon_precond_refresh_mx4(h, slot, 0, c, e, 1, 16, 4, 0.5f, nullptr) == MUON_ERR_BAD_ARG, "slot %d", slot);
  float* sums = nullptr;
  double* count = nullptr;
  int64_t ld = 0;
  CHECK(muon_precond_sums(h, 0, 0, &sums, &ld, &count) == MUON_OK && ld == 768 && sums && count, "sums");
  CHECK(reinterpret_cast<uintptr_t>(sums) % 256 == 0 && reinterpret_cast<uintptr_t>(sums) > (uintptr_t(1) << 40), "place");
  CHECK(muon_precond_sums(h, 0, 0, nullptr, nullptr, nullptr) == MUON_OK, "nothing asked for");
  CHECK(muon_precond_sums(h, 0, 1, &sums, &ld, &count) == MUON_ERR_BAD_ARG, "block");
  CHECK(muon_precond_sums(nullptr, 0, 0, &sums, &ld, &count) == MUON_ERR_NULL_ARG, "handle");
  (void)muon_destroy(h);
}

// No entry point lets an exception out, wherever an allocation or a launch fails.
static void check_mx4_exceptions() {
  Request r;
  muon_handle_t h = nullptr;
  if (r.init(&h) != MUON_OK) return (void)++g_bad;
  g_record = 0;
  uint8_t* const c = reinterpret_cast<uint8_t*>(uintptr_t(1) << 45);
  uint8_t* const e = reinterpret_cast<uint8_t*>(uintptr_t(1) << 46);
  std::vector<muon_mx4_t> list, bad;
  for (int k = 0; k < 90; ++k) list.push_back(matrix(k, 300, 200 + k, k % 2, true, true));
  bad = list;
  bad[77].col_scales = bad[5].col_scales;
  muon_mx4_t w = matrix(0, 768, 768, MUON_BF16, true, true);
  w.values = r.tensors[0].param;
  long_message();
  const struct { const char* name; std::function<muon_status_t()> call; } calls[] = {
      {"quantize", [&] { return muon_mx4_quantize(list.data(), 90, 0, 0, nullptr); }},
      {"quantize, overlapping", [&] { return muon_mx4_quantize(bad.data(), 90, 0, 0, nullptr); }},
      {"dequantize", [&] { return muon_mx4_dequantize(list.data(), 90, 0, nullptr); }},
      {"set_mx4_weights", [&] { return muon_set_mx4_weights(h, &w, 1); }},
      {"set_mx4_weights, others'", [&] { return muon_set_mx4_weights(h, list.data(), 90); }},
      {"step", [&] { return muon_step(h, -1.f, nullptr); }},
      {"accumulate", [&] { return muon_precond_accumulate_mx4(h, 0, 0, c, e, 64, 32, 4, 0.5, nullptr); }},
      {"refresh", [&] { return muon_precond_refresh_mx4(h, 0, 0, c, e, 64, 32, 4, 0.5f, nullptr); }},
      {"refresh, misaligned", [&] { return muon_precond_refresh_mx4(h, 0, 0, c + 1, e, 64, 32, 4, 0.5f, nullptr); }},
      {"sums, bad slot", [&] { return muon_precond_sums(h, 5, 0, nullptr, nullptr, nullptr); }},
  };
  for (hipError_t launch : {hipSuccess, hipErrorUnknown})
    for (const auto& call : calls)
      for (long k = 1; k < 64; ++k) {
        const long live = g_live;
        g_launch = launch;
        g_fail_at = k;
        try {
          const muon_status_t st = call.call();
          if (!g_fail_at && launch == hipErrorUnknown)
            CHECK(st != MUON_OK || std::string(call.name) == "set_mx4_weights", "%s: no error", call.name);
        } catch (...) {
          CHECK(false, "%s: an exception left the call at allocation %ld", call.name, k);
        }
        const bool reached = g_fail_at == 0;
        g_fail_at = 0;
        g_launch = hipSuccess;
        if (std::string(call.name) != "set_mx4_weights")
          CHECK(g_live <= live + 1, "%s: %ld allocations stay behind at %ld", call.name, g_live - live, k);   // the message
        if (!reached) break;
      }
  (void)muon_destroy(h);
}

int main(int argc, char** argv) {
  const std::string what = argc > 1 ? argv[1] : "";
  if (what == "launches") check_launches();
  else if (what == "weights") check_weights();
  else if (what == "acts") check_acts();
  else if (what == "exceptions") check_mx4_exceptions();
  else return 2;
  if (!g_bad) std::printf("ok\n");
  return g_bad ? 1 : 0;
}
