// Refusals of calls that need a device to get past their first checks. The program defines the
// HIP runtime calls of the library's host layer itself (its symbols come before the runtime's):
// one gfx950 device, two whose memory can be told apart, and launches that are only counted. No
// address is ever read. Each call has to be refused before the first launch, or, as it stands
// without the fault, has to reach one.
#include <hip/hip_runtime_api.h>

#include <cstdint>
#include <cstdio>
#include <cstring>
#include <functional>
#include <string>

#include "pmoe.h"

static int launches = 0, failures = 0;

// 16 MiB blocks: number i is device 0's, 64 + i device 1's, 128 + i the host's.
static char* block(int i, size_t at = 0) { return reinterpret_cast<char*>(((uintptr_t)i + 4096) << 24) + at; }

extern "C" {
hipError_t hipGetDevice(int* d) { return *d = 0, hipSuccess; }
hipError_t hipGetDeviceProperties(hipDeviceProp_t* p, int) {  // the header maps the name to its version
  std::memset(p, 0, sizeof *p);
  std::strcpy(p->gcnArchName, "gfx950:sramecc+:xnack-");
  return hipSuccess;
}
hipError_t hipPointerGetAttributes(hipPointerAttribute_t* a, const void* p) {
  const uintptr_t i = (reinterpret_cast<uintptr_t>(p) >> 24) - 4096;
  std::memset(a, 0, sizeof *a);
  if (i >= 128) return hipErrorInvalidValue;
  a->type = hipMemoryTypeDevice;
  a->device = i >= 64;
  return hipSuccess;
}
// what stands between <<<...>>> and the launch
hipError_t __hipPushCallConfiguration(dim3, dim3, size_t, hipStream_t) { return hipSuccess; }
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* lds, hipStream_t* s) {
  return *grid = *block = dim3(1), *lds = 0, *s = nullptr, hipSuccess;
}
hipError_t hipLaunchKernel(const void*, dim3, dim3, void**, size_t, hipStream_t) { return ++launches, hipSuccess; }
hipError_t hipGetLastError(void) { return hipSuccess; }
}

static void expect(const char* what, int rc, int want, const char* message = "") {
  const bool launched = launches > 0, refused = want != PMOE_OK;
  if (rc != want || launched == refused || std::string(pmoe_last_error()).find(message) == std::string::npos) {
    std::printf("FAIL %s: %d instead of %d, %d launches, last error: %s\n", what, rc, want, launches, pmoe_last_error());
    ++failures;
  }
  launches = 0;
}

// An argument, and what it may not share memory with.
static void each_shared(const char* what, std::initializer_list<void**> outputs, std::initializer_list<void**> others,
                        const std::function<int()>& call) {
  int i = 0;
  for (void** o : outputs)
    for (void** other : others) {
      if (o == other) continue;
      for (size_t at : {size_t(0), size_t(16)}) {
        void* keep = *o;
        *o = static_cast<char*>(*other) + at;
        expect((what + (" " + std::to_string(i))).c_str(), call(), PMOE_ERR_ARG, "overlaps");
        *o = keep;
      }
      ++i;
    }
  expect(what, call(), PMOE_OK);
}

// ---------------------------------------------------------------- adapters
struct Adapters {
  int T = 40, n = 12, H = 64, N = 48, R = 8;
  void *dy = block(0), *x = block(1), *v = block(2), *ids = block(3), *down = block(4), *up = block(5),
       *scale = block(6), *base = block(7), *out = block(8), *d_down = block(9), *d_up = block(10), *ws = block(11);
  int forward() const {
    return pmoe_adapter_forward(x, ids, PMOE_IDS_INT32, T, n, H, N, R, down, up, (float*)scale, base, out, (float*)v, ws,
                                1 << 24, nullptr);
  }
  int backward() const {
    return pmoe_adapter_backward(dy, x, (float*)v, ids, PMOE_IDS_INT32, T, n, H, N, R, down, up, (float*)scale, base,
                                 out, (float*)d_down, (float*)d_up, ws, 1 << 24, nullptr);
  }
};

static void adapters() {
  Adapters a;
  expect("backward", a.backward(), PMOE_OK);
  a.out = a.base = nullptr;  // the matrices' gradients alone; both matrices are read
  expect("backward without dx", a.backward(), PMOE_OK);
  a.down = nullptr;
  expect("no down", a.backward(), PMOE_ERR_POINTER, "down is null");
  a.down = block(128);
  expect("down on the host", a.backward(), PMOE_ERR_POINTER, "down is not");
  a.down = block(64);
  expect("down on another device", a.backward(), PMOE_ERR_POINTER, "down is on device 1");
}

static void adapters_apart() {
  Adapters f;
  const auto forward = [&] { return f.forward(); };
  each_shared("adapter_forward", {&f.v, &f.out}, {&f.x, &f.ids, &f.down, &f.up, &f.scale, &f.v, &f.out}, forward);
  f.ws = block(11);
  for (void** p : {&f.x, &f.ids, &f.down, &f.up, &f.scale, &f.base, &f.v, &f.out}) {
    f.ws = *p;
    expect("adapter_forward, ws", f.forward(), PMOE_ERR_ARG, "overlaps");
  }
  f.ws = block(11);
  f.v = f.base;
  expect("adapter_forward, v over base", f.forward(), PMOE_ERR_ARG, "overlaps");
  f.v = block(2), f.out = static_cast<char*>(f.base) + 64;
  expect("adapter_forward, some of base", f.forward(), PMOE_ERR_ARG, "overlaps");
  f.out = f.base;
  expect("adapter_forward in place", f.forward(), PMOE_OK);

  Adapters b;
  const auto backward = [&] { return b.backward(); };
  each_shared("adapter_backward", {&b.d_down, &b.d_up},
              {&b.dy, &b.x, &b.v, &b.ids, &b.down, &b.up, &b.scale, &b.base, &b.out, &b.d_down, &b.d_up}, backward);
  each_shared("adapter_backward, dx", {&b.out}, {&b.dy, &b.x, &b.v, &b.ids, &b.down, &b.up, &b.scale}, backward);
  for (void** p : {&b.dy, &b.x, &b.v, &b.ids, &b.down, &b.up, &b.scale, &b.base, &b.out, &b.d_down, &b.d_up}) {
    b.ws = *p;
    expect("adapter_backward, ws", b.backward(), PMOE_ERR_ARG, "overlaps");
  }
  b.ws = block(11), b.out = static_cast<char*>(b.base) + 64;
  expect("adapter_backward, some of base", b.backward(), PMOE_ERR_ARG, "overlaps");
  b.out = b.base;
  expect("adapter_backward in place", b.backward(), PMOE_OK);
  b.d_down = b.d_up = nullptr, b.out = b.x, b.base = nullptr;  // x and v are not read without the matrices' gradients
  expect("adapter_backward over what it does not read", b.backward(), PMOE_OK);
}

// ---------------------------------------------------------------- router
static void router() {
  const int T = 40, K = 2, E = 16, S = 12;  // every argument has more than 16 bytes
  void *logits = block(0), *ids = block(1), *off = block(2), *counts = block(3), *tokens = block(4), *prob = block(5),
       *balance = block(6), *z = block(7), *ws = block(8), *d_balance = block(9), *d_z = block(10), *d_w = block(11),
       *d_logits = block(12);
  each_shared("balance", {&counts, &tokens, &prob, &balance, &z, &ws},
              {&logits, &ids, &off, &counts, &tokens, &prob, &balance, &z, &ws}, [&] {
                return pmoe_router_balance((float*)logits, ids, PMOE_IDS_INT32, T, K, E, (int*)off, S, (int*)counts,
                                           (int*)tokens, (float*)prob, (float*)balance, (float*)z, ws, 1 << 20, nullptr);
              });
  const auto backward = [&] {
    return pmoe_router_backward((float*)logits, ids, PMOE_IDS_INT32, T, K, E, 0, (int*)off, S, (int*)counts, (int*)tokens,
                                (float*)d_balance, (float*)d_z, (float*)d_w, (float*)d_logits, nullptr);
  };
  each_shared("router_backward", {&d_logits}, {&ids, &off, &counts, &tokens, &d_balance, &d_z, &d_w}, backward);
  d_logits = static_cast<char*>(logits) + 64;
  expect("router_backward over some logits", backward(), PMOE_ERR_ARG, "overlaps");
  d_logits = logits;
  expect("router_backward in place", backward(), PMOE_OK);
  d_logits = d_w, d_balance = nullptr, counts = d_w, d_w = nullptr;  // counts are not read without d_balance
  expect("router_backward over what it does not read", backward(), PMOE_OK);
}

// ---------------------------------------------------------------- finalize
static void finalize() {
  void *dout = block(0), *z = block(1), *row = block(2), *w = block(3), *d_w = block(4), *d_z = block(5);
  const auto call = [&] {
    return pmoe_finalize_backward(dout, z, (int*)row, (float*)w, 40, 2, 64, 70, (float*)d_w, d_z, nullptr);
  };
  each_shared("finalize_backward", {&d_w, &d_z}, {&dout, &z, &row, &w, &d_w, &d_z}, call);
  d_z = nullptr, d_w = w;  // the weights are not read without d_z
  expect("finalize_backward over what it does not read", call(), PMOE_OK);
}

// What has no bytes overlaps nothing, wherever its pointer lies.
static void empty_ranges() {
  Adapters a;
  a.T = 0;
  a.dy = block(9, 64), a.x = block(10, 64), a.v = block(9, 128), a.ids = block(3), a.out = a.base = block(9, 256);
  expect("backward of no tokens, cut from the gradients' own memory", a.backward(), PMOE_OK);
  expect("gradients of no rows", pmoe_finalize_backward(block(0), block(0, 64), (int*)block(1), (float*)block(2), 4, 2, 64, 0,
                                                        (float*)block(3), block(0, 64), nullptr), PMOE_OK);
}

int main() {
  adapters();
  adapters_apart();
  router();
  finalize();
  empty_ranges();
  std::printf(failures ? "refusals: %d failures\n" : "refusals: ok\n", failures);
  return failures != 0;
}
