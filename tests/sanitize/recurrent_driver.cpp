// recurrent_driver.cpp -- host-side checks of the entry points in
// ssm_recurrent.h under AddressSanitizer and UndefinedBehaviorSanitizer (test
// infrastructure).
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

#include "ssm_recurrent.h"

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

const int64_t kEdge[] = {INT64_MIN, -1, 0, 1, 2, 15, 16, 17, 64, 65, 128, 4096, 65535, 65536, int64_t{1} << 22,
                         (int64_t{1} << 22) + 1, int64_t{1} << 31, int64_t{1} << 40, INT64_MAX};

}  // namespace

int main() {
  Blocks m;
  const hipStream_t s = nullptr;
  const auto f = [&] { return reinterpret_cast<float*>(m.get()); };
  void *x = m.get(), *r = m.get(), *i = m.get(), *z = m.get(), *out = m.get(), *dout = m.get();
  void *dx = m.get(), *dr = m.get(), *di = m.get(), *dz = m.get(), *ws = m.get();
  float *A = f(), *rb = f(), *ib = f(), *h0 = f(), *last = f(), *mid = f(), *dA = f(), *drb = f(), *dib = f(),
        *dh0 = f(), *dlast = f();
  int32_t* cu = reinterpret_cast<int32_t*>(m.get());
  char* const odd = static_cast<char*>(x) + 1;
  const size_t wsb = size_t{1} << 16;

  // ---- workspace queries over edge sizes (must never overflow) ----
  size_t acc = 0;
  for (int64_t b : kEdge)
    for (int64_t L : kEdge)
      for (int64_t d : kEdge) {
        for (int dt = -1; dt < 3; ++dt) {
          acc += ssm_gated_scan_fwd_workspace_bytes(b, L, d, dt);
          acc += ssm_gated_scan_fwd_varlen_workspace_bytes(b, L, d, dt);
          for (int have = 0; have < 2; ++have) {
            acc += ssm_gated_scan_bwd_workspace_bytes(b, L, d, dt, have);
            acc += ssm_gated_scan_bwd_varlen_workspace_bytes(b, L, d, dt, have);
          }
        }
        for (int64_t w : kEdge) {
          acc += ssm_causal_conv1d_bwd_workspace_bytes(b, L, d, w);
          for (int64_t h : kEdge) acc += ssm_qk_norm_rotate_bwd_workspace_bytes(b, L, h, w, d);
        }
      }
  std::printf("workspace queries done (%zu)\n", acc & 0xffff);

  // ---- gated scan: sizes, types, missing and misaligned pointers, overlaps, workspace ----
  const auto fwd = [&](int64_t b, int64_t L, int64_t d, int dt, int norm, const void* xx, void* o, void* w, size_t wb) {
    return ssm_gated_scan_fwd(xx, r, i, A, rb, ib, norm, z, o, last, h0, mid, b, L, d, dt, w, wb, s);
  };
  const auto fwd_v = [&](int64_t n, int64_t L, int64_t d, int dt, const int32_t* c, float* la, size_t wb) {
    return ssm_gated_scan_fwd_varlen(x, r, i, A, rb, ib, 1, z, out, la, h0, mid, c, n, L, d, dt, ws, wb, s);
  };
  const auto bwd = [&](int64_t b, int64_t L, int64_t d, int dt, const void* zz, void* dzz, float* dAA, size_t wb) {
    return ssm_gated_scan_bwd(x, r, i, A, rb, ib, 1, zz, h0, mid, dout, dlast, dx, dr, di, dzz, dAA, drb, dib, dh0, b,
                              L, d, dt, ws, wb, s);
  };
  const auto bwd_v = [&](int64_t n, int64_t L, int64_t d, const int32_t* c, size_t wb) {
    return ssm_gated_scan_bwd_varlen(x, r, i, A, rb, ib, 1, z, h0, nullptr, dout, dlast, dx, dr, di, dz, dA, drb, dib,
                                     dh0, c, n, L, d, 1, ws, wb, s);
  };
  for (int64_t v : kEdge) {
    if (v < 1 || v > (int64_t{1} << 22)) {
      expect(fwd(1, 8, v, 1, 1, x, out, ws, wsb), SSM_ERR_SHAPE, "fwd dim");
      expect(fwd_v(1, 8, v, 1, cu, last, wsb), SSM_ERR_SHAPE, "fwd varlen dim");
      expect(bwd(1, 8, v, 1, z, dz, dA, wsb), SSM_ERR_SHAPE, "bwd dim");
      expect(bwd_v(1, 8, v, cu, wsb), SSM_ERR_SHAPE, "bwd varlen dim");
    }
    if (v < 1 || v > 65535) {
      expect(fwd(v, 8, 8, 1, 1, x, out, ws, wsb), SSM_ERR_SHAPE, "fwd batch");
      expect(bwd(v, 8, 8, 1, z, dz, dA, wsb), SSM_ERR_SHAPE, "bwd batch");
    }
    if (v < 1 || v >= (int64_t{1} << 24)) {
      expect(fwd_v(v, 8, 8, 1, cu, last, wsb), SSM_ERR_SHAPE, "fwd nseq");
      expect(bwd_v(v, 8, 8, cu, wsb), SSM_ERR_SHAPE, "bwd nseq");
    }
    if (v < 0 || v > (int64_t{1} << 40)) expect(fwd(1, v, 8, 1, 1, x, out, ws, wsb), SSM_ERR_SHAPE, "fwd seqlen");
  }
  expect(fwd(1, 8, 8, 7, 1, x, out, ws, wsb), SSM_ERR_UNSUPPORTED, "fwd dtype");
  expect(fwd(1, 8, 8, 1, 2, x, out, ws, wsb), SSM_ERR_UNSUPPORTED, "fwd normalize");
  expect(fwd(1, 8, 8, 1, 1, nullptr, out, ws, wsb), SSM_ERR_NULL, "fwd x");
  expect(fwd(1, 8, 8, 1, 1, x, nullptr, ws, wsb), SSM_ERR_NULL, "fwd out");
  expect(fwd(1, 8, 8, 1, 1, odd, out, ws, wsb), SSM_ERR_ALIGN, "fwd x alignment");
  expect(fwd(1, 8, 8, 1, 1, x, r, ws, wsb), SSM_ERR_ALIAS, "fwd out over rgate");
  expect(fwd(1, 8, 8, 1, 1, x, mid, ws, wsb), SSM_ERR_ALIAS, "fwd out over chunk_states");
  expect(fwd(1, 600, 8, 1, 1, x, out, nullptr, 0), SSM_ERR_WORKSPACE, "fwd workspace");
  expect(fwd(1, 600, 8, 1, 1, x, out, ws, 16), SSM_ERR_WORKSPACE, "fwd workspace size");
  expect(fwd(1, 600, 8, 1, 1, x, out, static_cast<char*>(ws) + 8, wsb - 8), SSM_ERR_ALIGN, "fwd workspace alignment");
  expect(fwd_v(2, 8, 8, 1, nullptr, last, wsb), SSM_ERR_NULL, "fwd offsets");
  expect(fwd_v(2, 8, 8, 1, cu, h0, wsb), SSM_ERR_ALIAS, "varlen last over initial");
  expect(bwd(1, 8, 8, 1, z, nullptr, dA, wsb), SSM_ERR_NULL, "bwd dz");
  expect(bwd(1, 8, 8, 1, nullptr, dz, dA, wsb), SSM_ERR_NULL, "bwd dz without z");
  expect(bwd(1, 8, 8, 1, z, dz, nullptr, wsb), SSM_ERR_NULL, "bwd dA");
  expect(bwd(1, 8, 8, 1, z, dx, dA, wsb), SSM_ERR_ALIAS, "bwd dz over dx");
  expect(bwd(1, 8, 8, 1, z, dz, A, wsb), SSM_ERR_ALIAS, "bwd dA over A");
  expect(bwd(1, 8, 8, 1, z, dz, dA, 16), SSM_ERR_WORKSPACE, "bwd workspace size");
  expect(bwd_v(2, 8, 8, nullptr, wsb), SSM_ERR_NULL, "bwd offsets");
  expect(bwd_v(2, 8, 8, cu, 16), SSM_ERR_WORKSPACE, "bwd varlen workspace");

  // ---- step ----
  const auto step = [&](int64_t b, int64_t d, int dt, float* st, void* o) {
    return ssm_gated_state_update(st, x, r, i, A, rb, ib, 1, z, o, b, d, dt, s);
  };
  for (int64_t v : kEdge)
    if (v < 1 || v > (int64_t{1} << 31)) {
      expect(step(v, 8, 1, h0, out), SSM_ERR_SHAPE, "step batch");
      expect(step(8, v, 1, h0, out), SSM_ERR_SHAPE, "step dim");
    }
  expect(step(int64_t{1} << 31, int64_t{1} << 22, 1, h0, out), SSM_ERR_SHAPE, "step size");
  expect(step(1, 8, 3, h0, out), SSM_ERR_UNSUPPORTED, "step dtype");
  expect(step(1, 8, 1, nullptr, out), SSM_ERR_NULL, "step state");
  expect(step(1, 8, 1, h0, h0), SSM_ERR_ALIAS, "step out over state");

  // ---- norm with rotation ----
  const auto rot = [&](int64_t b, int64_t L, int64_t hq, int64_t hk, int64_t d, int64_t R, int64_t qs, int64_t ks,
                       float eps, int inter, int dt, const void* q, void* qo) {
    return ssm_qk_norm_rotate_fwd(q, r, A, rb, ib, cu, eps, inter, qo, dr, b, L, hq, hk, d, R, qs, ks, dt, s);
  };
  const auto rotb = [&](int64_t b, int64_t L, int64_t hq, int64_t hk, int64_t d, int64_t R, int64_t qs, int64_t ks,
                        const void* dq, void* w, size_t wb) {
    return ssm_qk_norm_rotate_bwd(x, r, A, rb, ib, cu, 1e-6f, 0, dq, z, dx, dr, dA, drb, b, L, hq, hk, d, R, qs, ks, 1,
                                  w, wb, s);
  };
  for (int64_t v : kEdge) {
    if (v < 2 || v > 256 || v % 2) {
      expect(rot(1, 2, 2, 1, v, 0, INT64_MAX / 2, INT64_MAX / 2, 0, 0, 1, x, out), SSM_ERR_UNSUPPORTED, "headdim");
    }
    if (v < 0 || v > 8 || v % 2) expect(rot(1, 2, 2, 1, 8, v, 16, 8, 0, 0, 1, x, out), SSM_ERR_UNSUPPORTED, "rotary_dim");
    if (v < 1 || v >= (int64_t{1} << 31)) expect(rot(v, 2, 2, 1, 8, 8, 16, 8, 0, 0, 1, x, out), SSM_ERR_SHAPE, "batch");
    if (v < 0 || v >= (int64_t{1} << 31)) expect(rotb(1, v, 2, 1, 8, 8, 16, 8, dout, ws, wsb), SSM_ERR_SHAPE, "seqlen");
    if (v < 1 || v > 65536) expect(rot(1, 2, v, 1, 8, 8, 16, 8, 0, 0, 1, x, out), SSM_ERR_SHAPE, "heads");
    if (v < 16 || v > (int64_t{1} << 30)) expect(rot(1, 2, 2, 1, 8, 8, v, 8, 0, 0, 1, x, out), SSM_ERR_SHAPE, "stride");
    if (v < 8 || v > (int64_t{1} << 30)) expect(rotb(1, 2, 2, 1, 8, 8, 16, v, dout, ws, wsb), SSM_ERR_SHAPE, "k stride");
  }
  expect(rot(1, 2, 2, 1, 8, 8, 16, 8, -1.0f, 0, 1, x, out), SSM_ERR_UNSUPPORTED, "eps");
  expect(rot(1, 2, 2, 1, 8, 8, 16, 8, std::nanf(""), 0, 1, x, out), SSM_ERR_UNSUPPORTED, "eps NaN");
  expect(rot(1, 2, 2, 1, 8, 8, 16, 8, 0, 2, 1, x, out), SSM_ERR_UNSUPPORTED, "interleaved");
  expect(rot(1, 2, 2, 1, 8, 8, 16, 8, 0, 0, 5, x, out), SSM_ERR_UNSUPPORTED, "dtype");
  expect(rot(1, 2, 2, 1, 8, 8, 16, 8, 0, 0, 1, nullptr, out), SSM_ERR_NULL, "q");
  expect(rot(1, 2, 2, 1, 8, 8, 16, 8, 0, 0, 1, odd, out), SSM_ERR_ALIGN, "q alignment");
  expect(rot(1, 2, 2, 1, 8, 8, 16, 8, 0, 0, 1, x, r), SSM_ERR_ALIAS, "q_out over k");
  expect(rot(1, 2, 2, 1, 8, 8, 24, 8, 0, 0, 1, x, x), SSM_ERR_ALIAS, "in place with a stride");
  expect(rot(1, 2, 2, 0, 8, 8, 16, 0, 0, 0, 1, x, out), SSM_ERR_NULL, "k without heads");
  expect(rotb(1, 2, 2, 1, 8, 8, 16, 8, nullptr, ws, wsb), SSM_ERR_NULL, "dq_out");
  expect(rotb(1, 2, 2, 1, 8, 8, 16, 8, dout, ws, 16), SSM_ERR_WORKSPACE, "rotate workspace");
  expect(rotb(1, 2, 2, 1, 8, 8, 16, 8, dx, ws, wsb), SSM_ERR_ALIAS, "dq over dq_out");

  // ---- convolution ----
  const auto conv = [&](int64_t b, int64_t L, int64_t d, int64_t w, int silu, int dt, void* o, size_t wb) {
    return ssm_causal_conv1d_bwd(x, A, rb, r, dout, i, o, dA, drb, di, b, L, d, w, silu, dt, ws, wb, s);
  };
  for (int64_t v : kEdge) {
    if (v < 2 || v > 4) expect(conv(1, 8, 8, v, 1, 1, dx, wsb), SSM_ERR_UNSUPPORTED, "width");
    if (v < 1 || v > 65535) expect(conv(v, 8, 8, 4, 1, 1, dx, wsb), SSM_ERR_SHAPE, "conv batch");
    if (v < 1 || v > (int64_t{1} << 22)) expect(conv(1, 8, v, 4, 1, 1, dx, wsb), SSM_ERR_SHAPE, "conv dim");
    if (v < 0 || v > (int64_t{1} << 31)) expect(conv(1, v, 8, 4, 1, 1, dx, wsb), SSM_ERR_SHAPE, "conv seqlen");
  }
  expect(conv(1, 8, 8, 4, 2, 1, dx, wsb), SSM_ERR_UNSUPPORTED, "silu");
  expect(conv(1, 8, 8, 4, 1, 9, dx, wsb), SSM_ERR_UNSUPPORTED, "conv dtype");
  expect(conv(1, 8, 8, 4, 1, 1, nullptr, wsb), SSM_ERR_NULL, "dx");
  expect(conv(1, 8, 8, 4, 1, 1, x, wsb), SSM_ERR_ALIAS, "dx over x");
  expect(conv(1, 8, 8, 4, 1, 1, dx, 16), SSM_ERR_WORKSPACE, "conv workspace");

  std::printf("%d call(s) not rejected\n", g_bad);
  return g_bad;
}
