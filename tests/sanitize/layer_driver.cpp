// layer_driver.cpp -- host-side checks of the entry points in ssm_layer.h under
// AddressSanitizer and UndefinedBehaviorSanitizer (test infrastructure).
//
// Every call carries an argument that the library must reject before it
// touches the device, and the workspace queries run over grids of edge and
// extreme sizes, where the size arithmetic would overflow if it were not
// checked.  Pointers are distinct host blocks: the host code compares their
// values (alignment, overlap) and must never dereference them.  Exit status:
// the number of calls that were not rejected.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "ssm_layer.h"

namespace {

int g_bad = 0;

void expect(int rc, int want, const char* what) {
  if (rc != want) {
    std::printf("NOT REJECTED AS %d (rc %d, \"%s\"): %s\n", want, rc, ssm_last_error(), what);
    ++g_bad;
  }
}

struct Blocks {
  std::vector<char*> v;
  char* get(size_t bytes = size_t{1} << 16) {
    char* p = static_cast<char*>(std::aligned_alloc(256, bytes));
    v.push_back(p);
    return p;
  }
  ~Blocks() {
    for (char* p : v) std::free(p);
  }
};

const int64_t kEdge[] = {INT64_MIN, -1, 0, 1, 2, 15, 16, 17, 64, 65, 256, 257, 65535, 65536, (int64_t{1} << 20) - 1,
                         int64_t{1} << 22, (int64_t{1} << 22) + 1, (int64_t{1} << 31) - 1, int64_t{1} << 31,
                         int64_t{1} << 40, INT64_MAX};
const int64_t kFew[] = {-1, 0, 1, 16, 256, 257, 65535, int64_t{1} << 31, INT64_MAX};

}  // namespace

int main() {
  Blocks m;
  const hipStream_t s = nullptr;
  const auto f = [&] { return reinterpret_cast<float*>(m.get()); };
  void *q = m.get(), *k = m.get(), *v = m.get(), *out = m.get(), *dout = m.get(), *ws = m.get(size_t{1} << 22);
  void *dq = m.get(), *dk = m.get(), *dv = m.get();
  float *beta = f(), *g = f(), *h0 = f(), *last = f(), *mid = f(), *dlast = f(), *dbeta = f(), *dg = f(), *dh0 = f();
  int32_t* cu = reinterpret_cast<int32_t*>(m.get());
  char* const odd = static_cast<char*>(q) + 1;
  const size_t wsb = size_t{1} << 22;

  // ---- workspace queries over edge sizes (must never overflow) ----
  size_t acc = 0;
  for (int64_t b : kEdge)
    for (int64_t L : kEdge) {
      for (int dt = -1; dt < 3; ++dt) acc += ssm_layer_norm_bwd_workspace_bytes(b, L, dt);
      for (int64_t hk : kFew)
        for (int64_t hv : kFew)
          for (int64_t K : kFew)
            for (int64_t V : kFew) {
              acc += ssm_delta_rule_fwd_workspace_bytes(b, L, hk, hv, K, V, 1);
              acc += ssm_delta_rule_fwd_varlen_workspace_bytes(b, L, hk, hv, K, V, 0);
              acc += ssm_delta_rule_bwd_workspace_bytes(b, L, hk, hv, K, V, 0, 0);
              acc += ssm_delta_rule_bwd_varlen_workspace_bytes(b, L, hk, hv, K, V, 1, 1);
            }
    }
  std::printf("workspace queries done (%zu)\n", acc & 0xffff);

  // ---- delta rule: sizes, strides, types, pointers, overlaps, workspace ----
  struct Sizes {
    int64_t n = 2, L = 40, hk = 1, hv = 2, K = 8, V = 4, qs = 8, ks = 8, vs = 8;
  };
  const auto fwd = [&](const Sizes& z, int dt, const void* qq, void* o, float* la, void* w, size_t wb) {
    return ssm_delta_rule_fwd(qq, k, v, beta, g, 1.0f, o, la, h0, mid, z.n, z.L, z.hk, z.hv, z.K, z.V, z.qs, z.ks, z.vs,
                              dt, w, wb, s);
  };
  const auto fwd_v = [&](const Sizes& z, const int32_t* c, float* la, size_t wb) {
    return ssm_delta_rule_fwd_varlen(q, k, v, beta, g, 1.0f, out, la, h0, mid, c, z.n, z.L, z.hk, z.hv, z.K, z.V, z.qs,
                                     z.ks, z.vs, 1, ws, wb, s);
  };
  const auto bwd = [&](const Sizes& z, int dt, const void* d, const float* gg, float* dgg, void* w, size_t wb) {
    return ssm_delta_rule_bwd(q, k, v, beta, gg, 1.0f, h0, mid, d, dlast, dq, dk, dv, dbeta, dgg, dh0, z.n, z.L, z.hk,
                              z.hv, z.K, z.V, z.qs, z.ks, z.vs, dt, w, wb, s);
  };
  const auto bwd_v = [&](const Sizes& z, const int32_t* c, size_t wb) {
    return ssm_delta_rule_bwd_varlen(q, k, v, beta, g, 1.0f, h0, mid, dout, dlast, dq, dk, dv, dbeta, dg, dh0, c, z.n,
                                     z.L, z.hk, z.hv, z.K, z.V, z.qs, z.ks, z.vs, 1, ws, wb, s);
  };
  const auto step = [&](const Sizes& z, int dt, float* st, void* o) {
    return ssm_delta_state_update(st, q, k, v, beta, g, 1.0f, o, z.n, z.hk, z.hv, z.K, z.V, z.qs, z.ks, z.vs, dt, s);
  };
  const auto all = [&](const Sizes& z, const char* what) {
    expect(fwd(z, 1, q, out, last, ws, wsb), SSM_ERR_SHAPE, what);
    expect(fwd_v(z, cu, last, wsb), SSM_ERR_SHAPE, what);
    expect(bwd(z, 1, dout, g, dg, ws, wsb), SSM_ERR_SHAPE, what);
    expect(bwd_v(z, cu, wsb), SSM_ERR_SHAPE, what);
  };
  for (int64_t x : kEdge) {
    Sizes z;
    z.n = x;
    if (x < 1 || x >= int64_t{1} << 22) all(z, "sequences");
    if (x < 1 || x >= int64_t{1} << 24) expect(step(z, 1, h0, out), SSM_ERR_SHAPE, "step batch");
    z = Sizes{}, z.L = x;
    if (x < 0 || x >= int64_t{1} << 31) all(z, "tokens");
    z = Sizes{}, z.hk = x;
    if (x < 1 || x > 2) all(z, "key heads"), expect(step(z, 1, h0, out), SSM_ERR_SHAPE, "step key heads");
    z = Sizes{}, z.hv = x;
    if (x < 1 || x > 2) all(z, "value heads or their stride");
    z = Sizes{}, z.K = x;
    if (x < 1 || x > 8) all(z, "headdim_k or its stride"), expect(step(z, 1, h0, out), SSM_ERR_SHAPE, "step headdim_k");
    z = Sizes{}, z.V = x, z.vs = int64_t{1} << 22;
    if (x < 1 || x > 256) all(z, "headdim_v"), expect(step(z, 1, h0, out), SSM_ERR_SHAPE, "step headdim_v");
    for (int which = 0; which < 3; ++which) {
      z = Sizes{};
      (which == 0 ? z.qs : which == 1 ? z.ks : z.vs) = x;
      if (x < 8 || x > int64_t{1} << 22) all(z, "stride"), expect(step(z, 1, h0, out), SSM_ERR_SHAPE, "step stride");
    }
  }
  const Sizes z;
  expect(fwd(z, 2, q, out, last, ws, wsb), SSM_ERR_UNSUPPORTED, "dtype");
  expect(fwd(z, 1, nullptr, out, last, ws, wsb), SSM_ERR_NULL, "q");
  expect(fwd(z, 1, odd, out, last, ws, wsb), SSM_ERR_ALIGN, "q alignment");
  expect(fwd(z, 1, q, k, last, ws, wsb), SSM_ERR_ALIAS, "out over k");
  expect(fwd(z, 1, q, out, beta, ws, wsb), SSM_ERR_ALIAS, "last over beta");
  expect(fwd(z, 1, q, out, h0 + 1, ws, wsb), SSM_ERR_ALIAS, "last partly over initial");
  expect(fwd(z, 1, q, out, last, ws, 16), SSM_ERR_WORKSPACE, "workspace size");
  expect(fwd(z, 1, q, out, last, nullptr, 0), SSM_ERR_WORKSPACE, "no workspace");
  expect(fwd(z, 1, q, out, last, static_cast<char*>(ws) + 8, wsb - 8), SSM_ERR_ALIGN, "workspace alignment");
  expect(fwd_v(z, nullptr, last, wsb), SSM_ERR_NULL, "offsets");
  expect(fwd_v(z, cu, reinterpret_cast<float*>(cu), wsb), SSM_ERR_ALIAS, "last over the offsets");
  expect(fwd_v(z, cu, last, 16), SSM_ERR_WORKSPACE, "varlen workspace");
  expect(bwd(z, 9, dout, g, dg, ws, wsb), SSM_ERR_UNSUPPORTED, "bwd dtype");
  expect(bwd(z, 1, nullptr, g, dg, ws, wsb), SSM_ERR_NULL, "dout");
  expect(bwd(z, 1, dout, nullptr, dg, ws, wsb), SSM_ERR_NULL, "dg without g");
  expect(bwd(z, 1, dq, g, dg, ws, wsb), SSM_ERR_ALIAS, "dq over dout");
  expect(bwd(z, 1, dout, g, g, ws, wsb), SSM_ERR_ALIAS, "dg over g");
  expect(bwd(z, 1, dout, g, dg, ws, 16), SSM_ERR_WORKSPACE, "bwd workspace size");
  expect(bwd_v(z, nullptr, wsb), SSM_ERR_NULL, "bwd offsets");
  expect(bwd_v(z, cu, 16), SSM_ERR_WORKSPACE, "bwd varlen workspace");
  expect(step(z, 3, h0, out), SSM_ERR_UNSUPPORTED, "step dtype");
  expect(step(z, 1, nullptr, out), SSM_ERR_NULL, "step state");
  expect(step(z, 1, h0, h0), SSM_ERR_ALIAS, "step out over state");

  // ---- layer norm ----
  const auto norm = [&](int64_t rows, int64_t dim, int64_t xs, int64_t rs, float eps, int dt, const void* x, void* o,
                        void* sum) {
    return ssm_layer_norm_fwd(x, k, beta, g, eps, o, sum, rows, dim, xs, rs, dt, s);
  };
  const auto normb = [&](int64_t rows, int64_t dim, int64_t ss, float eps, const void* d, void* dx, float* dw, size_t wb) {
    return ssm_layer_norm_bwd(q, beta, eps, d, k, dx, dw, dg, rows, dim, ss, 1, ws, wb, s);
  };
  for (int64_t x : kEdge) {
    if (x < 0 || x >= int64_t{1} << 31) {
      expect(norm(x, 8, 8, 8, 0, 1, q, out, dq), SSM_ERR_SHAPE, "rows");
      expect(normb(x, 8, 8, 0, dout, dq, dbeta, wsb), SSM_ERR_SHAPE, "bwd rows");
    }
    if (x < 1 || x > 16384) {
      expect(norm(4, x, int64_t{1} << 30, int64_t{1} << 30, 0, 1, q, out, dq), SSM_ERR_SHAPE, "dim");
      expect(normb(4, x, int64_t{1} << 30, 0, dout, dq, dbeta, wsb), SSM_ERR_SHAPE, "bwd dim");
    }
    if (x < 8 || x > int64_t{1} << 30) {
      expect(norm(4, 8, x, 8, 0, 1, q, out, dq), SSM_ERR_SHAPE, "x stride");
      expect(norm(4, 8, 8, x, 0, 1, q, out, dq), SSM_ERR_SHAPE, "residual stride");
      expect(normb(4, 8, x, 0, dout, dq, dbeta, wsb), SSM_ERR_SHAPE, "s stride");
    }
  }
  expect(norm(4, 8, 8, 8, -1.0f, 1, q, out, dq), SSM_ERR_UNSUPPORTED, "eps");
  expect(norm(4, 8, 8, 8, std::nanf(""), 1, q, out, dq), SSM_ERR_UNSUPPORTED, "eps NaN");
  expect(norm(4, 8, 8, 8, 0, 5, q, out, dq), SSM_ERR_UNSUPPORTED, "norm dtype");
  expect(norm(4, 8, 8, 8, 0, 1, nullptr, out, dq), SSM_ERR_NULL, "x");
  expect(norm(4, 8, 8, 8, 0, 1, odd, out, dq), SSM_ERR_ALIGN, "x alignment");
  expect(norm(4, 8, 8, 8, 0, 1, q, out, out), SSM_ERR_ALIAS, "sum over out");
  expect(norm(4, 8, 16, 8, 0, 1, q, q, dq), SSM_ERR_ALIAS, "in place with a stride");
  expect(normb(4, 8, 8, 0, nullptr, dq, dbeta, wsb), SSM_ERR_NULL, "norm dout");
  expect(normb(4, 8, 8, 0, dout, q, dbeta, wsb), SSM_ERR_ALIAS, "dx over s");
  expect(normb(4, 8, 8, 0, dout, dq, beta, wsb), SSM_ERR_ALIAS, "dweight over weight");
  expect(normb(4, 8, 8, 0, dout, dq, dbeta, 16), SSM_ERR_WORKSPACE, "norm workspace");

  std::printf("%d call(s) not rejected\n", g_bad);
  return g_bad;
}
