// Which launches on lists of 4-bit matrices go past the caches: by the bytes of
// their values, not by the tiles that hold them.  Prints "ok".
#include <cstdio>
#include <cstring>
#include <initializer_list>

#include "muon_internal.h"

static int g_bad = 0;
#define CHECK(x) (void)((x) || (std::printf("line %d: %s\n", __LINE__, #x), ++g_bad))

struct Size { int32_t rows, cols; };
static muon::Mx4List list(std::initializer_list<Size> sizes) {
  muon::Mx4List l;
  std::memset(&l, 0x5A, sizeof(l));           // nothing behind the last matrix counts
  l.n = l.tiles = 0;
  for (const Size& x : sizes) {
    muon::Mx4Dev& m = l.m[l.n++];
    m.rows = x.rows;
    m.cols = x.cols;
    m.tiles_c = (x.cols + 127) / 128;
    l.tiles += (x.rows + 127) / 128 * m.tiles_c;
  }
  return l;
}

int main() {
  using muon::mx4_round_streams;
  // 4 MB and 8 MB in one row or one column: of the 256 MB that a launch is streamed from, whatever their tiles
  for (Size x : {Size{1, 1 << 21}, Size{1 << 21, 1}}) {
    CHECK(int64_t(list({x}).tiles) * 128 * 128 * 2 > int64_t(256) << 20);
    CHECK(!mx4_round_streams(list({x}), false) && !mx4_round_streams(list({x}), true));
  }
  CHECK(!mx4_round_streams(list({{8192, 16384}}), false) && mx4_round_streams(list({{8193, 16384}}), false));
  CHECK(!mx4_round_streams(list({{8192, 8192}}), true) && mx4_round_streams(list({{8193, 8192}}), true));
  CHECK(!mx4_round_streams(list({{8192, 8192}, {4096, 16384}}), false));
  CHECK(mx4_round_streams(list({{8192, 8192}, {4096, 16384}, {1, 1}}), false));
  CHECK(mx4_round_streams(list({{1, 1 << 30}}), true) && mx4_round_streams(list({{1 << 30, 1}, {1 << 30, 1}}), true));
  // read back: from 4 MB of values on
  using muon::mx4_back_streams;
  CHECK(!mx4_back_streams(list({{1, 768}}), false) && !mx4_back_streams(list({{1, 1 << 20}}), true));
  CHECK(!mx4_back_streams(list({{1024, 1024}, {1024, 1024}}), false));
  CHECK(mx4_back_streams(list({{1024, 1024}, {1024, 1024}, {1, 1}}), false) && mx4_back_streams(list({{1025, 1024}}), true));
  if (!g_bad) std::puts("ok");
  return g_bad != 0;
}
