// The host side of the row operators (rows.hip) and of the products in 8 bits
// (i8.hip) with the kernel launches replaced by lines on stdout, so that plans,
// workspace sizes and refusals can be tested without a GPU.  One call per line
// of stdin:
//   entry name=value ...   (fields of the entry's descriptor)
// Prints the launches of the call, then "status <s> query <s> need <bytes>" of
// the call and of its size query (where it has one).
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

#include "../implicit_gemm_convolution_amd/csrc/i8.hip"
#include "../implicit_gemm_convolution_amd/csrc/rows.hip"

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
template <bool BF, int MODE>
int launch_product(const igc_ffn::GemmArgs& args, const Plan& pl, hipStream_t) {
  const auto& a = static_cast<const igc_ffn::I8Args&>(args);
  std::printf("product mode=%d variant=%d odd=%d M=%d N=%d R=%d lda=%lld ldb=%lld whole=%lld splits=%d groups=%lld part=%zu a=%llu b=%llu\n", MODE,
              pl.variant, a.odd_rows, a.M, a.N, a.R, a.lda, a.ldb, pl.whole, pl.splits, workgroups(pl), pl.part_bytes,
              (unsigned long long)reinterpret_cast<uintptr_t>(a.A), (unsigned long long)reinterpret_cast<uintptr_t>(a.B));
  return IGC_OK;
}
#define DEFINE(n, BF, MODE) template int launch_product<BF, MODE>(const igc_ffn::GemmArgs&, const Plan&, hipStream_t);
IGC_I8_KINDS(DEFINE)
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
    if (entry == "linear_i8") {
      igc_linear_i8 d{};
      I(M); I(N); I(K); I(act); I(y_type); P(X); I(ldx); P(x_scale); P(W); I(ldw); P(w_scale); P(bias); P(R); I(ldr); P(Y); I(ldy);
      P(workspace); d.ws_bytes = f("ws_bytes");
      both(d, linear_i8, linear_i8_workspace_size);
    } else if (entry == "glu_i8") {
      igc_glu_i8 d{};
      I(M); I(N); I(K); I(type); I(act); P(X); I(ldx); P(x_scale); P(Wg); I(ldwg); P(wg_scale); P(Wu); I(ldwu); P(wu_scale); P(bias_g);
      P(bias_u); P(H); I(ldh); P(workspace); d.ws_bytes = f("ws_bytes");
      both(d, glu_i8, glu_i8_workspace_size);
    } else if (entry == "layer_norm_backward") {
      igc_layer_norm_backward d{};
      I(M); I(N); I(type); I(x_type); P(dY); I(lddy); P(X); I(ldx); P(mean); P(rstd); P(gamma); P(R); I(ldr); P(dX); I(lddx); P(dgamma);
      P(dbeta); P(workspace); d.ws_bytes = f("ws_bytes");
      both(d, layer_norm_backward, layer_norm_backward_workspace_size);
    } else if (entry == "layer_norm_forward") {
      igc_layer_norm_forward d{};
      I(M); I(N); I(type); I(x_type); P(X); I(ldx); P(Y); I(ldy); P(Q); I(ldq); P(scale);
      const int s = layer_norm_forward(&d, nullptr);
      std::printf("status %d query 0 need 0 %s\n", s, s ? g_error : "");
    } else {
      std::printf("unknown entry %s\n", entry.c_str());
      return 1;
    }
  }
  return 0;
}
