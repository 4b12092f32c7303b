// Host-side status plumbing shared by every libfl entry point.
#include <stdarg.h>
#include <string.h>

#include "fl_kv.cuh"

namespace fl {

static thread_local char g_msg[1024] = "";

void set_error(const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_msg, sizeof(g_msg), fmt, ap);
  va_end(ap);
}

fl_status fail(fl_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_msg, sizeof(g_msg), fmt, ap);
  va_end(ap);
  return st;
}

fl_status cuda_fail(cudaError_t e, const char* what) {
  snprintf(g_msg, sizeof(g_msg), "%s: %s", what, cudaGetErrorString(e));
  return FL_ERR_CUDA;
}

int device_sm_count() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  static int cache[64] = {0};
  if (dev >= 0 && dev < 64 && cache[dev] > 0) return cache[dev];
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  if (dev >= 0 && dev < 64) cache[dev] = n;
  return n;
}

}  // namespace fl

extern "C" const char* fl_status_string(int status) {
  switch (status) {
    case FL_OK: return "FL_OK";
    case FL_ERR_ARG: return "FL_ERR_ARG";
    case FL_ERR_SHAPE: return "FL_ERR_SHAPE";
    case FL_ERR_UNSUPPORTED: return "FL_ERR_UNSUPPORTED";
    case FL_ERR_ALIGN: return "FL_ERR_ALIGN";
    case FL_ERR_CUDA: return "FL_ERR_CUDA";
    case FL_ERR_WORKSPACE: return "FL_ERR_WORKSPACE";
    case FL_ERR_TIMEOUT: return "FL_ERR_TIMEOUT";
    default: return "FL_ERR_UNKNOWN";
  }
}

extern "C" const char* fl_last_error(void) { return fl::g_msg; }

extern "C" int fl_version(void) { return 1; }

namespace fl {
namespace gemv {
int take_device_error();
}
namespace kq {
int take_device_error();
}
namespace tc {
int take_device_error();
}
namespace kv {
int take_device_error();
}
namespace attn {
int take_device_error();
}
namespace attn_tc {
int take_device_error();
}
int take_gate_error();
}  // namespace fl

extern "C" fl_status fl_device_status(void) {
  using namespace fl;
  FL_CHECK_CUDA(cudaDeviceSynchronize(), "fl_device_status: cudaDeviceSynchronize");
  const int g = gemv::take_device_error(), k = kq::take_device_error(), t = take_gate_error();
  const int c = tc::take_device_error(), v = kv::take_device_error(), a1 = attn::take_device_error();
  const int a2 = attn_tc::take_device_error();
  if (g < 0 || k < 0 || t < 0 || c < 0 || v < 0 || a1 < 0 || a2 < 0)
    return fail(FL_ERR_CUDA, "fl_device_status: reading the error words failed");
  const int at = a1 | a2;
  if (g == 0 && k == 0 && t == 0 && c == 0 && v == 0 && at == 0) return FL_OK;
  // Every word was cleared, so every pending error is named; a wait that ran out decides the status.
  char msg[sizeof(g_msg)] = "";
  bool timeout = false;
  auto add = [&](bool wait, const char* fmt, auto... args) {
    timeout = timeout || wait;
    size_t n = strlen(msg);
    if (n > 0 && n + 2 < sizeof(msg)) n += strlen(strcpy(msg + n, "; "));
    snprintf(msg + n, sizeof(msg) - n, fmt, args...);
  };
  auto what = [](int c) {
    return c == 1 ? "a producer's wait for a free stage" : c == 2 ? "a consumer's wait for a full stage"
         : c == 3 ? "the wait for staged activations" : c == 4 ? "the self-test wait" : "a wait";
  };
  if (g && g != 5) add(true, "plane GEMV: %s ran out (code %d); its outputs are not valid", what(g), g);
  if (k) add(true, "K-quant GEMV: %s ran out (code %d); its outputs are not valid", what(k), k);
  if (c) {
    const char* cw = c == 1 ? "the producer's wait for a free stage" : c == 2 ? "the MMA issuer's wait for codes or a free accumulator"
                   : c == 3 ? "a converter's wait for a full stage or a free code buffer" : "an epilogue wait for the MMAs";
    add(true, "tensor-core GEMV: %s ran out (code %d); its outputs are not valid", cw, c);
  }
  if (t) add(true, "logit gate: the wait for the cluster's partials ran out; its outputs are NaN");
  if (at & kv::kErrWait) add(true, "attention: a wait ran out; its outputs are not valid");
  if (g == 5) add(false, "plane GEMV: a listed block index was out of range; that unit was skipped");
  for (const auto& e : {std::make_pair(v, "cache append or read"), std::make_pair(at, "attention")}) {
    if (e.first & kv::kErrPage) add(false, "%s: a page index was out of range; that block was left out", e.second);
    if (e.first & kv::kErrSeq)
      add(false, "%s: a sequence's length or rows contradict the batch; it was left out", e.second);
  }
  return fail(timeout ? FL_ERR_TIMEOUT : FL_ERR_ARG, "%s", msg);
}
