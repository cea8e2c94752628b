// Host-side checks of the attention side of libqlora under the address and
// undefined-behaviour sanitizers (host code instrumented, no GPU needed): each
// entry point's refusals, the workspace queries over many shapes, and what a
// call that is accepted hands to its kernels.  The launchers are replaced at
// link time (-Wl,--wrap) by ones that record their arguments, so nothing here
// reaches a GPU and no address given is ever read.  Exit status 0 means every
// expectation held.
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "kernels.hpp"
#include "kvcache.hpp"
#include "qlora.h"

using qlora::AttendProblem;

static int failures = 0, launches = 0;
static AttendProblem attended;

#define EXPECT(cond)                                              \
  do {                                                            \
    if (!(cond)) {                                                \
      fprintf(stderr, "FAILED line %d: %s\n", __LINE__, #cond);   \
      ++failures;                                                 \
    }                                                             \
  } while (0)
#define REFUSED(call, status)          \
  do {                                 \
    const int before_ = launches;      \
    EXPECT((call) == (status));        \
    EXPECT(launches == before_);       \
  } while (0)
#define LAUNCHED(call)                 \
  do {                                 \
    const int before_ = launches;      \
    EXPECT((call) == QLORA_OK);        \
    EXPECT(launches == before_ + 1);   \
  } while (0)

extern "C" {
hipError_t __wrap__ZN5qlora13launch_attendERKNS_13AttendProblemEPKfPvP12ihipStream_t(const AttendProblem& p, const float*,
                                                                                     void*, hipStream_t) {
  attended = p;
  ++launches;
  return hipSuccess;
}
hipError_t __wrap__ZN5qlora11launch_ropeEliRKNS_9RopeTableEbRKNS_9HeadsViewES5_S5_S5_P12ihipStream_t(
    int64_t, int32_t, const qlora::RopeTable&, bool, const qlora::HeadsView&, const qlora::HeadsView&,
    const qlora::HeadsView&, const qlora::HeadsView&, hipStream_t) {
  ++launches;
  return hipSuccess;
}
hipError_t __wrap__ZN5qlora17launch_rope_tableERKNS_13RopeTableArgsEPfP12ihipStream_t(const qlora::RopeTableArgs&, float*,
                                                                                      hipStream_t) {
  ++launches;
  return hipSuccess;
}
hipError_t __wrap__ZN5qlora15launch_kv_writeERKNS_6KVPoolElRKNS_9HeadsViewES5_PKlRKNS_9RopeTableERKNS_9MidpointsEP12ihipStream_t(
    const qlora::KVPool&, int64_t, const qlora::HeadsView&, const qlora::HeadsView&, const int64_t*, const qlora::RopeTable&,
    const qlora::Midpoints&, hipStream_t) {
  ++launches;
  return hipSuccess;
}
hipError_t __wrap__ZN5qlora14launch_kv_readERKNS_6KVPoolElPKlPtS5_PKfP12ihipStream_t(const qlora::KVPool&, int64_t,
                                                                                      const int64_t*, uint16_t*, uint16_t*,
                                                                                      const float*, hipStream_t) {
  ++launches;
  return hipSuccess;
}
}

template <typename T>
static T* at(uintptr_t a) {
  return reinterpret_cast<T*>(a);
}
static const uintptr_t kAddr = 0x10000;

static qlora_heads heads(int32_t n = 4, int64_t token = 256, int64_t head = 64, uintptr_t data = kAddr) {
  return qlora_heads{at<uint16_t>(data), token, head, n};
}
static qlora_kv_cache cache(int32_t type = QLORA_KV_INT8, int32_t n = 4, int32_t dim = 64, int32_t page = 16,
                            int64_t pages = 10) {
  return qlora_kv_cache{at<void>(kAddr), at<void>(kAddr), at<float>(kAddr), at<float>(kAddr), pages, type, n, dim, page};
}

static void check_rope_table() {
  struct Args {
    int64_t n = 8;
    int32_t rot = 64;
    double base = 1e4;
    int32_t scaling = QLORA_ROPE_NONE;
    double factor = 1, original = 0, low = 1, high = 32, amplitude = 1;
    float* table = at<float>(kAddr);
    int run() const {
      return qlora_rope_table(n, rot, base, scaling, factor, original, low, high, amplitude, table, nullptr);
    }
  };
  const double inf = __builtin_inf(), nan = __builtin_nan("");
  Args a;
  LAUNCHED(a.run());
  for (int32_t rot : {0, 8, 24, 272, -16}) { a = Args(); a.rot = rot; REFUSED(a.run(), QLORA_ERR_UNSUPPORTED); }
  for (double x : {0.0, -1.0, inf, nan}) {
    a = Args(); a.base = x; REFUSED(a.run(), QLORA_ERR_UNSUPPORTED);
    a = Args(); a.amplitude = x; REFUSED(a.run(), QLORA_ERR_UNSUPPORTED);
    a = Args(); a.scaling = QLORA_ROPE_LINEAR; a.factor = x; REFUSED(a.run(), QLORA_ERR_UNSUPPORTED);
  }
  for (int32_t s : {-1, 4, INT32_MAX}) { a = Args(); a.scaling = s; REFUSED(a.run(), QLORA_ERR_UNSUPPORTED); }
  a = Args(); a.scaling = QLORA_ROPE_BANDS; a.factor = 2; REFUSED(a.run(), QLORA_ERR_UNSUPPORTED);
  a.original = 4096; LAUNCHED(a.run());
  a.low = 32; REFUSED(a.run(), QLORA_ERR_UNSUPPORTED);
  for (int64_t n : {int64_t(-1), INT64_MIN, INT64_MAX}) { a = Args(); a.n = n; REFUSED(a.run(), QLORA_ERR_SHAPE); }
  a = Args(); a.table = nullptr; REFUSED(a.run(), QLORA_ERR_NULL);
  a.n = 0; REFUSED(a.run(), QLORA_OK);
  a = Args(); a.table = at<float>(kAddr + 4); REFUSED(a.run(), QLORA_ERR_ALIGN);
}

static void check_rope() {
  struct Args {
    int64_t T = 3;
    int32_t dim = 64, rot = 64, inter = 0, inverse = 0;
    const float* table = at<float>(kAddr);
    int64_t n = 16;
    const int32_t* pos = at<int32_t>(kAddr);
    qlora_heads q = heads(), qo = heads(), k = heads(2), ko = heads(2);
    bool with_k = true, with_ko = true;
    int run() const {
      return qlora_rope(T, dim, rot, inter, inverse, table, n, pos, &q, &qo, with_k ? &k : nullptr, with_ko ? &ko : nullptr,
                        nullptr);
    }
  };
  Args a;
  LAUNCHED(a.run());
  a.with_k = a.with_ko = false; LAUNCHED(a.run());
  a.with_k = true; REFUSED(a.run(), QLORA_ERR_NULL);
  for (int32_t d : {0, 8, 72, 272, -16}) { a = Args(); a.dim = d; REFUSED(a.run(), QLORA_ERR_UNSUPPORTED); }
  for (int32_t r : {0, 24, 80, -16}) { a = Args(); a.rot = r; REFUSED(a.run(), QLORA_ERR_UNSUPPORTED); }
  a = Args(); a.inter = 2; REFUSED(a.run(), QLORA_ERR_UNSUPPORTED);
  a = Args(); a.inverse = -1; REFUSED(a.run(), QLORA_ERR_UNSUPPORTED);
  for (int64_t n : {int64_t(-1), INT64_MIN, INT64_MAX}) {
    a = Args(); a.T = n; REFUSED(a.run(), QLORA_ERR_SHAPE);
    a = Args(); a.n = n; REFUSED(a.run(), QLORA_ERR_SHAPE);
  }
  a = Args(); a.T = 0; a.table = nullptr; REFUSED(a.run(), QLORA_OK);
  a = Args(); a.table = nullptr; REFUSED(a.run(), QLORA_ERR_NULL);
  a = Args(); a.pos = nullptr; REFUSED(a.run(), QLORA_ERR_NULL);
  a = Args(); a.q.data = nullptr; REFUSED(a.run(), QLORA_ERR_NULL);
  a = Args(); a.q.data = at<uint16_t>(kAddr + 8); REFUSED(a.run(), QLORA_ERR_ALIGN);
  a = Args(); a.q.token_stride = 255; REFUSED(a.run(), QLORA_ERR_ALIGN);
  a = Args(); a.qo.head_stride = 60; REFUSED(a.run(), QLORA_ERR_ALIGN);
  for (int32_t h : {0, -1, INT32_MIN, INT32_MAX}) { a = Args(); a.q.heads = a.qo.heads = h; REFUSED(a.run(), QLORA_ERR_SHAPE); }
  // Strides of more than 2^32 elements, the one whose magnitude int64 cannot hold among them.
  for (int64_t s : {INT64_MIN, -(int64_t(1) << 33), int64_t(1) << 33, INT64_MAX - 7}) {
    a = Args(); a.q.token_stride = s; REFUSED(a.run(), QLORA_ERR_SHAPE);
    a = Args(); a.ko.head_stride = s; REFUSED(a.run(), QLORA_ERR_SHAPE);
  }
  a = Args(); a.q.token_stride = -(int64_t(1) << 32); a.k.head_stride = int64_t(1) << 32; LAUNCHED(a.run());
  a = Args(); a.qo.heads = 5; REFUSED(a.run(), QLORA_ERR_SHAPE);
  a = Args(); a.ko.heads = 5; REFUSED(a.run(), QLORA_ERR_SHAPE);
}

static void check_cache() {
  struct Args {
    qlora_kv_cache c = cache();
    int64_t T = 3;
    qlora_heads k = heads(), v = heads();
    const int64_t* slots = at<int64_t>(kAddr);
    const float* table = nullptr;
    int64_t n = 0;
    const int32_t* pos = nullptr;
    int32_t rot = 0, inter = 0;
    int write() const { return qlora_kv_write(&c, T, &k, &v, slots, table, n, pos, rot, inter, nullptr); }
    int read() const { return qlora_kv_read(&c, T, slots, k.data, v.data, nullptr); }
  };
  Args a;
  for (int32_t type : {QLORA_KV_BF16, QLORA_KV_INT8, QLORA_KV_NF4, QLORA_KV_INT4, QLORA_KV_FP4}) {
    a = Args(); a.c.type = type;
    LAUNCHED(a.write());
    LAUNCHED(a.read());
    a.c.k_scale = nullptr;
    if (type == QLORA_KV_BF16) { LAUNCHED(a.write()); LAUNCHED(a.read()); }
    else { REFUSED(a.write(), QLORA_ERR_NULL); REFUSED(a.read(), QLORA_ERR_NULL); }
  }
#define BOTH(status) do { REFUSED(a.write(), status); REFUSED(a.read(), status); a = Args(); } while (0)
  a = Args();
  for (int32_t t : {-1, 5, INT32_MAX}) { a.c.type = t; BOTH(QLORA_ERR_UNSUPPORTED); }
  for (int32_t d : {0, 40, 512, -16}) { a.c.dim = d; BOTH(QLORA_ERR_UNSUPPORTED); }
  for (int32_t p : {0, 8, 24, 2048, INT32_MIN, -16}) { a.c.page_size = p; BOTH(QLORA_ERR_UNSUPPORTED); }
  for (int32_t h : {0, -1, INT32_MIN, INT32_MAX}) { a.c.heads = h; BOTH(QLORA_ERR_SHAPE); }
  for (int64_t p : {int64_t(0), int64_t(-1), INT64_MIN, INT64_MAX}) { a.c.pages = p; BOTH(QLORA_ERR_SHAPE); }
  for (int64_t t : {int64_t(-1), INT64_MIN, INT64_MAX}) { a.T = t; BOTH(QLORA_ERR_SHAPE); }
  a.c.k = nullptr; BOTH(QLORA_ERR_NULL);
  a.c.v = at<void>(kAddr + 8); BOTH(QLORA_ERR_ALIGN);
  a.c.v_scale = at<float>(kAddr + 4); BOTH(QLORA_ERR_ALIGN);
  a.slots = nullptr; BOTH(QLORA_ERR_NULL);
  a.slots = at<int64_t>(kAddr + 4); BOTH(QLORA_ERR_ALIGN);
  a.v.data = nullptr; BOTH(QLORA_ERR_NULL);
  a.k.data = at<uint16_t>(kAddr + 2); BOTH(QLORA_ERR_ALIGN);
  a.T = 0; a.slots = nullptr; BOTH(QLORA_OK);
#undef BOTH
  REFUSED(qlora_kv_write(nullptr, 3, &a.k, &a.v, a.slots, nullptr, 0, nullptr, 0, 0, nullptr), QLORA_ERR_NULL);
  REFUSED(qlora_kv_read(nullptr, 3, a.slots, a.k.data, a.v.data, nullptr), QLORA_ERR_NULL);
  a.v.heads = 3; REFUSED(a.write(), QLORA_ERR_SHAPE);
  a = Args(); a.table = at<float>(kAddr); a.pos = at<int32_t>(kAddr); a.n = 8; a.rot = 64;
  LAUNCHED(a.write());
  for (int32_t r : {0, 24, 80}) { a.rot = r; REFUSED(a.write(), QLORA_ERR_UNSUPPORTED); }
  a.rot = 64; a.n = 0; REFUSED(a.write(), QLORA_ERR_SHAPE);
  a.n = 8; a.pos = nullptr; REFUSED(a.write(), QLORA_ERR_NULL);
}

struct Attend {
  qlora_kv_cache c = cache();
  int64_t tokens = 8;
  qlora_heads q = heads();
  int32_t batch = 2;
  const int32_t* pages = at<int32_t>(kAddr);
  int64_t width = 4;
  const int32_t* starts = at<int32_t>(kAddr);
  const int32_t* lengths = at<int32_t>(kAddr);
  int64_t max_new = 4, max_len = 64;
  float scale = 0.1f;
  int32_t causal = 1;
  int64_t window = 0;
  uint16_t* out = at<uint16_t>(kAddr);
  float* lse = nullptr;
  void* ws = at<void>(kAddr);
  size_t ws_bytes = size_t(1) << 40;
  int run() const {
    return qlora_attend_paged(&c, tokens, &q, batch, pages, width, starts, lengths, max_new, max_len, scale, causal, window,
                              out, lse, ws, ws_bytes, nullptr);
  }
  size_t need() const {
    return qlora_attend_paged_workspace_bytes(&c, tokens, q.heads, batch, max_new, max_len, causal, window);
  }
};

static void check_attend() {
  Attend a;
  LAUNCHED(a.run());
  EXPECT(attended.width == 4 && attended.max_len == 64 && attended.max_new == 4);
#define BAD(status) do { REFUSED(a.run(), status); a = Attend(); } while (0)
  a.c.dim = 24; BAD(QLORA_ERR_UNSUPPORTED);
  for (int64_t x : {int64_t(-1), INT64_MIN}) {
    a.tokens = x; BAD(QLORA_ERR_SHAPE);
    a.max_new = x; BAD(QLORA_ERR_SHAPE);
    a.max_len = x; BAD(QLORA_ERR_SHAPE);
    a.window = x; BAD(QLORA_ERR_SHAPE);
    a.width = x; BAD(QLORA_ERR_SHAPE);
  }
  a.tokens = INT64_MAX; BAD(QLORA_ERR_SHAPE);
  a.max_len = INT64_MAX; BAD(QLORA_ERR_SHAPE);
  for (int64_t w : {INT64_MAX, int64_t(1) << 60, int64_t(1) << 59, (int64_t(1) << 30) + 1}) { a.width = w; BAD(QLORA_ERR_SHAPE); }
  a.batch = -1; BAD(QLORA_ERR_SHAPE);
  a.batch = 1 << 17; BAD(QLORA_ERR_SHAPE);
  a.max_len = 65; BAD(QLORA_ERR_SHAPE);
  for (int32_t h : {0, 6, -4, INT32_MAX}) { a.q.heads = h; BAD(QLORA_ERR_SHAPE); }
  a.causal = 2; BAD(QLORA_ERR_UNSUPPORTED);
  a.scale = __builtin_inff(); BAD(QLORA_ERR_UNSUPPORTED);
  a.pages = nullptr; BAD(QLORA_ERR_NULL);
  a.starts = nullptr; BAD(QLORA_ERR_NULL);
  a.lengths = nullptr; BAD(QLORA_ERR_NULL);
  a.out = nullptr; BAD(QLORA_ERR_NULL);
  a.q.data = nullptr; BAD(QLORA_ERR_NULL);
  a.out = at<uint16_t>(kAddr + 8); BAD(QLORA_ERR_ALIGN);
  a.lse = at<float>(kAddr + 2); BAD(QLORA_ERR_ALIGN);
  a.q.token_stride = 4; BAD(QLORA_ERR_ALIGN);
  a.tokens = 0; a.starts = nullptr; BAD(QLORA_OK);
#undef BAD
  a.tokens = a.batch = 1; a.max_new = 1; a.max_len = 4096; a.width = 256;
  const size_t need = a.need();
  EXPECT(need > 0);
  a.ws_bytes = need; LAUNCHED(a.run());
  a.ws_bytes = need - 1; REFUSED(a.run(), QLORA_ERR_WORKSPACE);
  a.ws_bytes = need; a.ws = nullptr; REFUSED(a.run(), QLORA_ERR_WORKSPACE);
  a.ws = at<void>(kAddr + 4); REFUSED(a.run(), QLORA_ERR_ALIGN);
  a.c.dim = 24; EXPECT(a.need() == 0);
}

// Nothing is stored: no table of pages is needed, however many pages a sequence
// may have, and the kernels are told of no entry that they could read.
static void check_nothing_stored() {
  for (int64_t width : {0, 1, 4, 1000})
    for (int64_t window : {0, 5})
      for (int64_t n : {1, 100}) {
        Attend a;
        a.pages = nullptr;
        a.width = width;
        a.max_len = 0;
        a.window = window;
        a.tokens = 2 * n;
        a.max_new = n;
        LAUNCHED(a.run());
        EXPECT(attended.width == 0 && attended.max_len == 0);
        a.pages = at<int32_t>(kAddr);
        LAUNCHED(a.run());
        EXPECT(attended.width == 0);
      }
}

// A query over many shapes: it answers (0 or a size), and a size is enough for
// the call of the same shape.
static void check_workspace() {
  for (int32_t type = 0; type < 5; ++type)
    for (int32_t dim : {16, 80, 128, 256})
      for (int32_t group : {1, 8})
        for (int32_t h : {1, 8, 52})
          for (int64_t batch : {1, 3, 64})
            for (int64_t n : {1, 5, 40, 4096})
              for (int64_t len : {0, 1, 63, 4096, 8178, 131072})
                for (int64_t window : {0, 700}) {
                  Attend a;
                  a.c = cache(type, h, dim);
                  a.q = heads(h * group);
                  a.batch = (int32_t)batch;
                  a.tokens = batch * n;
                  a.max_new = n;
                  a.max_len = len;
                  a.window = window;
                  a.width = (len + 15) / 16;
                  a.ws_bytes = a.need();
                  if (!a.ws_bytes) a.ws = nullptr;
                  LAUNCHED(a.run());
                }
}

// Keys are split for the sake of parallel work alone: not because they are many,
// and never into splits that no row reaches.  So a prompt that fills the chip
// needs no workspace at any length, and what the kernel for many rows (more than
// 32 per key/value head) needs has a bound that no length enters: the splits of
// fewer row tiles than the chip holds (1024 of 128 rows, or 512 of 256), at most
// twice as many in all, each row's sums in fp32.
static void check_workspace_growth() {
  for (int64_t n : {4096, 8177, 8178, 8192, 16384, 32768, 131072}) {
    for (int32_t type : {QLORA_KV_BF16, QLORA_KV_INT8, QLORA_KV_NF4}) {
      Attend a;
      a.c = cache(type, 52, 128);
      a.q = heads(52);
      a.batch = 1;
      a.tokens = a.max_new = a.max_len = n;
      EXPECT(a.need() == 0);
      a.c = cache(type, 8, 128);
      a.q = heads(64);
      if (n >= 16384) EXPECT(a.need() == 0);
    }
  }
  for (int32_t type = 0; type < 5; ++type)
    for (int32_t dim : {16, 64, 128, 256})
      for (int32_t group : {1, 8})
        for (int32_t h : {1, 8, 52})
          for (int64_t batch : {1, 4, 64})
            for (int64_t n : {40, 129, 4096, 20000})
              for (int64_t len : {20000, 131072, 1 << 20, 1 << 30})
                for (int64_t window : {0, 700, 100000}) {
                  Attend a;
                  a.c = cache(type, h, dim);
                  a.q = heads(h * group);
                  a.batch = (int32_t)batch;
                  a.tokens = batch * n;
                  a.max_new = n;
                  a.max_len = len;
                  a.window = window;
                  EXPECT(a.need() <= (size_t)2 * 1024 * 128 * (dim + 2) * 4 + 256);
                }
  // One split of 16384 keys for few rows, where there is work enough.
  Attend a;
  a.c = cache(QLORA_KV_BF16, 8, 128);
  a.q = heads(64);
  a.batch = 256;
  a.tokens = 256;
  a.max_new = 1;
  a.max_len = 16384;
  EXPECT(a.need() == 0);
}

// Launches of 2^32 threads and more lose the upper bits of their count: refused.
static void check_grid_limits() {
  EXPECT(qlora_rope_table(int64_t(1) << 30, 16, 1e4, 0, 1, 0, 1, 32, 1, at<float>(kAddr), nullptr) == QLORA_ERR_SHAPE);
  LAUNCHED(qlora_rope_table((int64_t(1) << 29) - 64, 16, 1e4, 0, 1, 0, 1, 32, 1, at<float>(kAddr), nullptr));
  REFUSED(qlora_rope_table(int64_t(1) << 26, 128, 1e4, 0, 1, 0, 1, 32, 1, at<float>(kAddr), nullptr), QLORA_ERR_SHAPE);
  const qlora_heads h8 = heads(8, 1024, 128), h2 = heads(2, 1024, 128);
  auto rope = [&](int64_t T) {
    return qlora_rope(T, 128, 128, 0, 0, at<float>(kAddr), 8, at<int32_t>(kAddr), &h8, &h8, &h8, &h8, nullptr);
  };
  REFUSED(rope(int64_t(1) << 25), QLORA_ERR_SHAPE);         // 16 heads of 8 units
  REFUSED(rope((int64_t(1) << 25) + 5), QLORA_ERR_SHAPE);
  LAUNCHED(rope((int64_t(1) << 25) - 4));
  qlora_kv_cache c = cache(QLORA_KV_NF4, 2, 128);
  auto write = [&](int64_t T) {
    return qlora_kv_write(&c, T, &h2, &h2, at<int64_t>(kAddr), nullptr, 0, nullptr, 0, 0, nullptr);
  };
  auto read = [&](int64_t T) {
    return qlora_kv_read(&c, T, at<int64_t>(kAddr), at<uint16_t>(kAddr), at<uint16_t>(kAddr), nullptr);
  };
  REFUSED(write(int64_t(1) << 28), QLORA_ERR_SHAPE);        // keys and values, one group of heads, 8 lanes
  REFUSED(write(int64_t(1) << 30), QLORA_ERR_SHAPE);
  LAUNCHED(write((int64_t(1) << 28) - 32));
  REFUSED(read(int64_t(1) << 27), QLORA_ERR_SHAPE);         // keys and values of 2 heads, 8 units
  REFUSED(read((int64_t(1) << 27) + 1), QLORA_ERR_SHAPE);
  LAUNCHED(read((int64_t(1) << 27) - 16));
  Attend a;
  a.c = cache(QLORA_KV_BF16, 256, 64);
  a.q = heads(256);
  a.batch = 65535;
  a.tokens = 65535;
  a.max_new = 1;
  LAUNCHED(a.run());                                        // 65535 * 256 workgroups of 256
  a.c.heads = a.q.heads = 512;
  REFUSED(a.run(), QLORA_ERR_SHAPE);
  a.max_new = 16;                                           // as many workgroups, of more rows
  a.tokens = 65535 * 16;
  REFUSED(a.run(), QLORA_ERR_SHAPE);
  a.c = cache(QLORA_KV_INT8, 128, 64);                      // 256-row tiles take 512 threads
  a.q = heads(128);
  a.max_new = 200;
  a.tokens = 65535 * 200;
  a.max_len = 64;
  LAUNCHED(a.run());
  a.max_new = 300;
  a.tokens = 65535 * 300;
  REFUSED(a.run(), QLORA_ERR_SHAPE);
}

int main() {
  check_rope_table();
  check_rope();
  check_cache();
  check_attend();
  check_nothing_stored();
  check_workspace();
  check_workspace_growth();
  check_grid_limits();
  if (failures) {
    fprintf(stderr, "%d expectation(s) failed\n", failures);
    return 1;
  }
  printf("generate_asan: all host checks passed (%d launches recorded)\n", launches);
  return 0;
}
