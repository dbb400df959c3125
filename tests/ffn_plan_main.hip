// The host side of the feed-forward entry points (ffn.hip) with the kernel
// launches replaced by lines on stdout, so that plans, workspace sizes and
// refusals can be tested without a GPU.  One call per line of stdin:
//   entry name=value ...   (fields of the entry's descriptor)
// Prints the launches of the call, then "status <s> need <bytes>" of the call
// and of its size query.
#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdio>
#include <iostream>
#include <map>
#include <sstream>
#include <string>

static char g_error[256];
static void launched(const char* kernel, dim3 grid, dim3 threads) {
  std::printf("launch %s groups=%u threads=%u\n", kernel, grid.x, threads.x);
}
#undef hipLaunchKernelGGL
#define hipLaunchKernelGGL(kernel, grid, threads, lds, stream, ...) launched(#kernel, grid, threads)
#define hipGetLastError() hipSuccess

#include "../implicit_gemm_convolution_amd/csrc/ffn.hip"

namespace igc_host {
int fail(int status, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(g_error, sizeof(g_error), fmt, ap);
  va_end(ap);
  return status;
}
int check_device(int* dev) {
  *dev = 0;
  return IGC_OK;
}
int device_cus(int) { return 256; }
}  // namespace igc_host

namespace igc_ffn_host {
static void print(const char* name, int mode, const igc_ffn::GemmArgs& a, const Plan& pl) {
  std::printf("%s mode=%d variant=%d odd=%d M=%d N=%d R=%d whole=%lld splits=%d groups=%lld part=%zu\n", name, mode, pl.variant,
              a.odd_rows, a.M, a.N, a.R, pl.whole, pl.splits, workgroups(pl), pl.part_bytes);
}
template <bool BF, int MODE>
int launch_product(const igc_ffn::GemmArgs& a, const Plan& pl, hipStream_t) {
  print("product", MODE, a, pl);
  return IGC_OK;
}
template <bool BF>
int launch_back(const igc_ffn::GemmArgs& x, const Plan& px, const igc_ffn::GemmArgs& w, const Plan& pw, const igc_ffn::ColsumArgs&,
                hipStream_t) {
  print("joint", igc_ffn::M_DX, x, px);
  print("joint", igc_ffn::M_DW, w, pw);
  return IGC_OK;
}
#define DEFINE(n, BF, MODE) template int launch_product<BF, MODE>(const igc_ffn::GemmArgs&, const Plan&, hipStream_t);
IGC_FFN_KINDS(DEFINE)
template int launch_back<false>(const igc_ffn::GemmArgs&, const Plan&, const igc_ffn::GemmArgs&, const Plan&, const igc_ffn::ColsumArgs&,
                                hipStream_t);
template int launch_back<true>(const igc_ffn::GemmArgs&, const Plan&, const igc_ffn::GemmArgs&, const Plan&, const igc_ffn::ColsumArgs&,
                               hipStream_t);
}  // namespace igc_ffn_host

struct Fields {
  std::map<std::string, long long> v;
  long long operator()(const char* k) const {
    const auto i = v.find(k);
    return i == v.end() ? 0 : i->second;
  }
  template <class T>
  T* p(const char* k) const {
    return reinterpret_cast<T*>(static_cast<uintptr_t>((*this)(k)));
  }
};
#define I(k) d.k = (int)f(#k)
#define P(k) d.k = f.p<std::remove_pointer_t<decltype(d.k)>>(#k)

template <class D, class Q>
static void both(const D& d, int (*call)(const D*, void*), Q query) {
  size_t need = 0;
  const int q = query(&d, &need), c = call(&d, nullptr);
  std::printf("status %d query %d need %zu %s\n", c, q, need, c || q ? g_error : "");
}

int main() {
  std::string line, entry, word;
  while (std::getline(std::cin, line)) {
    std::istringstream in(line);
    in >> entry;
    Fields f;
    while (in >> word) f.v[word.substr(0, word.find('='))] = std::stoll(word.substr(word.find('=') + 1), nullptr, 0);
    if (entry == "linear_forward") {
      igc_linear_forward d{};
      I(M); I(N); I(K); I(type); I(act); I(y_type); P(X); I(ldx); P(W); I(ldw); P(bias); P(R); I(ldr); P(Y); I(ldy); P(Z); I(ldz);
      P(workspace); d.ws_bytes = f("ws_bytes");
      both(d, linear_forward, linear_forward_workspace_size);
    } else if (entry == "linear_backward") {
      igc_linear_backward d{};
      I(M); I(N); I(K); I(type); I(act); P(dY); I(lddy); P(Z); I(ldz); P(X); I(ldx); P(W); I(ldw); P(dX); I(lddx); P(dW); I(lddw);
      P(dbias); P(workspace); d.ws_bytes = f("ws_bytes");
      both(d, linear_backward, linear_backward_workspace_size);
    } else if (entry == "glu_forward") {
      igc_glu_forward d{};
      I(M); I(N); I(K); I(type); I(act); P(X); I(ldx); P(Wg); I(ldwg); P(Wu); I(ldwu); P(bias_g); P(bias_u); P(H); I(ldh); P(G);
      I(ldg); P(U); I(ldu); P(workspace); d.ws_bytes = f("ws_bytes");
      both(d, glu_forward, glu_forward_workspace_size);
    } else if (entry == "glu_backward") {
      igc_glu_backward d{};
      I(M); I(N); I(K); I(type); I(act); P(dH); I(lddh); P(G); I(ldg); P(U); I(ldu); P(X); I(ldx); P(Wg); I(ldwg); P(Wu); I(ldwu);
      P(dX); I(lddx); P(dWg); I(lddwg); P(dWu); I(lddwu); P(dbias_g); P(dbias_u); P(workspace); d.ws_bytes = f("ws_bytes");
      both(d, glu_backward, glu_backward_workspace_size);
    } else {
      std::printf("unknown entry %s\n", entry.c_str());
      return 1;
    }
  }
  return 0;
}
