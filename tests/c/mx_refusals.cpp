// Refusals of the permutation and the microscaled calls that need a device to get past their first
// checks, with the HIP runtime calls of the library's host layer defined here, as in refusals.cpp: one
// gfx950 device, another whose memory can be told apart, launches that are only counted. No address
// is ever read.
#include <hip/hip_runtime_api.h>

#include <cstdint>
#include <cstdio>
#include <cstring>
#include <functional>
#include <string>
#include <vector>

#include "pmoe.h"

static int launches = 0, failures = 0;

// 16 MiB blocks: number i is device 0's, 64 + i device 1's, 128 + i the host's.
static char* block(int i, size_t at = 0) { return reinterpret_cast<char*>(((uintptr_t)i + 4096) << 24) + at; }

extern "C" {
hipError_t hipGetDevice(int* d) { return *d = 0, hipSuccess; }
hipError_t hipGetDeviceProperties(hipDeviceProp_t* p, int) {
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
hipError_t __hipPushCallConfiguration(dim3, dim3, size_t, hipStream_t) { return hipSuccess; }
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* lds, hipStream_t* s) {
  return *grid = *block = dim3(1), *lds = 0, *s = nullptr, hipSuccess;
}
hipError_t hipLaunchKernel(const void*, dim3, dim3, void**, size_t, hipStream_t) { return ++launches, hipSuccess; }
hipError_t hipGetLastError(void) { return hipSuccess; }
}

static void expect(const std::string& what, int rc, int want, const char* message = "") {
  const bool launched = launches > 0, refused = want != PMOE_OK;
  if (rc != want || launched == refused || std::string(pmoe_last_error()).find(message) == std::string::npos) {
    std::printf("FAIL %s: %d instead of %d, %d launches, last error: %s\n", what.c_str(), rc, want, launches,
                pmoe_last_error());
    ++failures;
  }
  launches = 0;
}

struct Arg {
  const char* name;
  void** p;
  size_t align;
  int null_rc = PMOE_ERR_POINTER;
};

// Every pointer null, on the host, on another device and off its alignment; every output on every other argument.
static void pointers(const std::string& call, const std::vector<Arg>& outputs, const std::vector<Arg>& inputs,
                     const std::function<int()>& f) {
  expect(call, f(), PMOE_OK);
  std::vector<Arg> all = outputs;
  all.insert(all.end(), inputs.begin(), inputs.end());
  for (const Arg& a : all) {
    void* keep = *a.p;
    const std::string what = call + ", " + a.name;
    *a.p = nullptr;
    expect(what + " null", f(), a.null_rc, a.name);
    *a.p = block(130);
    expect(what + " on the host", f(), PMOE_ERR_POINTER, a.name);
    *a.p = block(70);
    expect(what + " on device 1", f(), PMOE_ERR_POINTER, "is on device 1");
    if (a.align > 1) {
      *a.p = static_cast<char*>(keep) + a.align / 2;
      expect(what + " misaligned", f(), PMOE_ERR_POINTER, a.name);
    }
    *a.p = keep;
  }
  for (const Arg& o : outputs)
    for (const Arg& other : all) {
      if (o.p == other.p) continue;
      void* keep = *o.p;
      *o.p = *other.p;
      expect(call + ", " + o.name + " over " + other.name, f(), PMOE_ERR_ARG, "overlaps");
      *o.p = keep;
    }
}

static void permutation() {
  const int T = 40, K = 4, E = 8;
  void *ids = block(0), *x = block(1), *rows = block(2), *row = block(3), *route = block(4), *off = block(5), *ws = block(6);
  const size_t need = pmoe_permute_workspace_bytes(T, K, E);
  size_t have = need;
  const auto f = [&] {
    return pmoe_permute_tokens(ids, PMOE_IDS_INT64, T, K, E, 0, x, 128, rows, (int*)row, (int*)route, (int*)off, ws, have,
                               nullptr);
  };
  pointers("permute_tokens", {{"rows", &rows, 16, PMOE_ERR_ARG}, {"row_of_route", &row, 4}, {"route_of_row", &route, 4},
                              {"expert_offsets", &off, 4}, {"ws", &ws, 256}},
           {{"topk_ids", &ids, 8}, {"x", &x, 16, PMOE_ERR_ARG}}, f);  // x and rows: both or neither
  have = need - 1;
  expect("permute_tokens, small workspace", f(), PMOE_ERR_WORKSPACE, "workspace too small");
  have = need;
  // the end of one argument on the start of another, and just behind it
  rows = static_cast<char*>(x) + T * 128 - 16;
  expect("permute_tokens, rows on the last bytes of x", f(), PMOE_ERR_ARG, "overlaps");
  rows = static_cast<char*>(x) + T * 128;
  expect("permute_tokens, rows behind x", f(), PMOE_OK);
  x = rows = nullptr;
  expect("permute_tokens without rows", f(), PMOE_OK);
  expect("no tokens", pmoe_permute_tokens(nullptr, PMOE_IDS_INT32, 0, K, E, 0, nullptr, 0, nullptr, nullptr, nullptr,
                                          (int*)off, ws, need, nullptr), PMOE_OK);

  void *d = block(1), *dx = block(2);
  pointers("permute_tokens_backward", {{"dx", &dx, 16}}, {{"d_rows", &d, 16}, {"row_of_route", &row, 4}}, [&] {
    return pmoe_permute_tokens_backward(d, PMOE_BF16, (int*)row, T, K, T * K, 64, dx, nullptr);
  });
  expect("gradient of no rows", pmoe_permute_tokens_backward(nullptr, PMOE_F32, (int*)row, T, K, 0, 64, dx, nullptr), PMOE_OK);
}

static void formats() {
  void *x = block(0), *codes = block(1), *sf = block(2);
  for (int format : {PMOE_MX_E2M1, PMOE_MX_E4M3})
    for (int type : {PMOE_BF16, PMOE_F32}) {
      const std::string what = " " + std::to_string(format) + std::to_string(type);
      pointers("mx_quantize" + what, {{"codes", &codes, 16}, {"scales", &sf, 1}}, {{"x", &x, 16}},
               [&] { return pmoe_mx_quantize(x, type, format, 16, 64, codes, sf, nullptr); });
      pointers("mx_dequantize" + what, {{"out", &x, 16}}, {{"codes", &codes, 16}, {"scales", &sf, 1}},
               [&] { return pmoe_mx_dequantize(codes, sf, format, 16, 64, type, x, nullptr); });
    }
}

static void products() {
  void *a = block(0), *a_sf = block(1), *route = block(2), *off = block(3), *w = block(4), *w_sf = block(5), *out = block(6);
  int R = 64, rows = 64, Kd = 256;
  bool gather = false;
  const auto f = [&] {
    return pmoe_mx_grouped_gemm(a, a_sf, rows, gather ? (int*)route : nullptr, 2, (int*)off, R, 4, w, w_sf, 64, Kd, out,
                                PMOE_BF16, nullptr);
  };
  pointers("mx_grouped_gemm", {{"out", &out, 16}},
           {{"a_codes", &a, 16}, {"a_sf", &a_sf, 4}, {"expert_offsets", &off, 4}, {"w_codes", &w, 16}, {"w_sf", &w_sf, 4}}, f);
  gather = true, rows = 32;
  out = route;
  expect("mx_grouped_gemm, out over route_of_row", f(), PMOE_ERR_ARG, "overlaps");
  out = block(6);
  expect("mx_grouped_gemm, gathered", f(), PMOE_OK);
  rows = 0, a = a_sf = nullptr;
  expect("mx_grouped_gemm of no tokens", f(), PMOE_OK);
  rows = 32, a = block(0), a_sf = block(1, 1), w_sf = block(5, 3), Kd = 96;  // rows of scales that are no whole dwords
  expect("mx_grouped_gemm, scales by bytes", f(), PMOE_OK);

  void *dy = block(0), *dx = block(6);
  w_sf = block(5);
  pointers("mx_grouped_gemm_backward", {{"dx", &dx, 16}},
           {{"dy", &dy, 16}, {"expert_offsets", &off, 4}, {"w_codes", &w, 16}, {"w_sf", &w_sf, 4}},
           [&] { return pmoe_mx_grouped_gemm_backward(dy, (int*)off, 64, 4, w, w_sf, 64, 256, dx, nullptr); });
}

static void activations() {
  void *y = block(0), *count = block(1), *hq = block(2), *h_sf = block(3), *y8 = block(4), *y8_sf = block(5), *dh = block(6),
       *dy = block(7);
  for (int act : {PMOE_ACT_RELU2, PMOE_ACT_SWIGLU}) {
    pointers("mx_activation", {{"hq", &hq, 16}, {"h_sf", &h_sf, 1}}, {{"y", &y, 16}}, [&] {
      return pmoe_mx_activation(y, 40, 64, act, 0.0f, (int*)count, hq, h_sf, y8, y8_sf, nullptr);
    });
    // y8 and y8_sf, where they are wanted
    const auto keep = [&] { return pmoe_mx_activation(y, 40, 64, act, 0.0f, nullptr, hq, h_sf, y8, y8_sf, nullptr); };
    y8 = block(70);
    expect("mx_activation, y8 on device 1", keep(), PMOE_ERR_POINTER, "y8 is on device 1");
    y8 = block(4, 8);
    expect("mx_activation, y8 misaligned", keep(), PMOE_ERR_POINTER, "y8");
    for (void* other : {y, hq, h_sf, y8_sf}) {
      y8 = other;
      expect("mx_activation, y8 over another", keep(), PMOE_ERR_ARG, "overlaps");
    }
    y8 = y8_sf = nullptr;
    expect("mx_activation without a checkpoint", keep(), PMOE_OK);
    y8 = block(4), y8_sf = block(5);
    expect("mx_activation, count on the host",
           pmoe_mx_activation(y, 40, 64, act, 0.0f, (int*)block(130), hq, h_sf, y8, y8_sf, nullptr), PMOE_ERR_POINTER, "row_count");
    expect("mx_activation, codes over the count",
           pmoe_mx_activation(y, 40, 64, act, 0.0f, (int*)hq, hq, h_sf, y8, y8_sf, nullptr), PMOE_ERR_ARG, "overlaps");
    pointers("mx_activation_backward", {{"dy", &dy, 16}}, {{"dh", &dh, 16}, {"y8", &y8, 16}, {"y8_sf", &y8_sf, 1}}, [&] {
      return pmoe_mx_activation_backward(dh, y8, y8_sf, 40, 64, act, 0.0f, nullptr, dy, nullptr);
    });
  }
}

int main() {
  permutation();
  formats();
  products();
  activations();
  std::printf(failures ? "refusals: %d failures\n" : "refusals: ok\n", failures);
  return failures != 0;
}
