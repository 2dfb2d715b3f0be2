// CPU check of the channels-last backward's plans: the workspace holds what a
// call from any source lays out in it, the staged kernels get only rows whose
// distances their 32-bit steps hold, the aligned copies read no byte outside
// their tensor, and the generic filter gradient chains few additions.
#include <cstdio>
#include "nhwc_bwd.h"

namespace dwconv {
// what the planner's file calls in others; nothing here is launched
cudaError_t bwd_weight_pass2(const Conv&, const float*, int, void*, void*, cudaStream_t) { return cudaErrorNotSupported; }
const char* algo_name(Algo) { return ""; }
namespace nhwc {
namespace walk {
#define X(T)                                                                                                          \
  template <>                                                                                                         \
  cudaError_t run<T>(const Conv&, const Geom&, bool, const T*, const Act8&, const T*, const T*, T*, float*, cudaStream_t) { \
    return cudaErrorNotSupported;                                                                                     \
  }                                                                                                                   \
  template <>                                                                                                         \
  cudaError_t run_staged<T>(const Conv&, const Staged&, int, const Views&, const Act8&, const T*, T*, float*,         \
                            cudaStream_t) {                                                                           \
    return cudaErrorNotSupported;                                                                                     \
  }
X(float) X(__half) X(__nv_bfloat16)
#undef X
}  // namespace walk
}  // namespace nhwc
}  // namespace dwconv
#include "nhwc_bwd.cu"

using namespace dwconv;
static int fails = 0, checks = 0, tall = 0;

static Conv mk(int64_t N, int64_t C, int64_t H, int64_t W, int k, int s, int p, int dtype) {
  Conv c{};
  c.N = N; c.C = C; c.H = H; c.W = W; c.m = 1; c.kh = c.kw = k; c.sh = c.sw = s; c.ph = c.pw = p; c.dh = c.dw = 1;
  c.Ho = (H + 2 * p - k) / s + 1; c.Wo = (W + 2 * p - k) / s + 1;
  c.off = 0; c.ctot = C; c.dtype = dtype;
  return c;
}

// every source's sums and aligned copies lie inside the workspace
static void check_room(const Conv& c) {
  const int es = c.dtype == DWCONV_F32 ? 4 : 2;
  const size_t size = nhwc::bwd_workspace_bytes(c);
  bool staged[2];
  for (int i = 0; i < 2; ++i) {
    nhwc::walk::Staged g;
    staged[i] = nhwc::walk::plan_staged(c, i ? kSrcI8 : kSrcFull, &g) && nhwc::copies_fit(c, es);
    if (!staged[i]) continue;
    const size_t copies = (size_t)(nhwc::gy_copy_bytes(c, es) + nhwc::x_copy_bytes(c, i ? 1 : es));
    const size_t sums = nhwc::sums_bytes(c, copies ? nhwc::walk_chunks(c) : g.chunks);
    ++checks;
    if (sums + copies > size) {
      ++fails;
      printf("FAIL %s N=%lld C=%lld H=%lld W=%lld k=%d s=%d: %zu of sums and %zu of copies in %zu\n", i ? "codes" : "full",
             (long long)c.N, (long long)c.C, (long long)c.H, (long long)c.W, c.kh, c.sh, sums, copies, size);
    }
  }
  tall += staged[0] != staged[1];
}

// rows whose scales (blocks of 32) are 2^32 bytes apart or more are not staged from codes
static void check_rows(const Conv& c, bool from_codes) {
  nhwc::walk::Staged g;
  const bool full = nhwc::walk::plan_staged(c, kSrcFull, &g), codes = nhwc::walk::plan_staged(c, kSrcI8, &g);
  ++checks;
  if (full && codes == from_codes) return;
  ++fails;
  printf("FAIL N=%lld C=%lld H=%lld W=%lld: staged from full values %d, from codes %d\n", (long long)c.N, (long long)c.C,
         (long long)c.H, (long long)c.W, (int)full, (int)codes);
}

// the aligned copies' reads: inside the tensor, each byte of a pixel brought
static uint8_t arena[4096];
static const uint8_t *inside_lo, *inside_end;
static bool outside;
struct Recorded {
  static uint32_t word(const uint8_t* p) {
    if (p < inside_lo || p + 4 > inside_end || (uintptr_t)p % 4) outside = true;
    return (uint32_t)p[0] | (uint32_t)p[1] << 8 | (uint32_t)p[2] << 16 | (uint32_t)p[3] << 24;
  }
  static uint32_t byte(const uint8_t* p) {
    if (p < inside_lo || p >= inside_end) outside = true;
    return *p;
  }
};
static void check_reads(int offset, int pixels, int from, int bytes) {
  inside_lo = arena + 64 + offset;
  inside_end = inside_lo + (pixels - 1) * from + bytes;
  outside = false;
  bool same = true;
  for (int p = 0; p < pixels; ++p)
    for (int at = 0; at < bytes; at += 16) {
      const uint8_t* src = inside_lo + p * from + at;
      uint32_t v[5];
      nhwc::words_at<Recorded>(src, inside_lo, inside_end, v);
      const int shift = (int)((uintptr_t)src & 3);
      for (int b = 0; b < 16 && at + b < bytes; ++b)
        same &= (uint8_t)(v[(b + shift) / 4] >> (8 * ((b + shift) % 4))) == src[b];
    }
  ++checks;
  if (outside || !same) {
    ++fails;
    printf("FAIL reads at offset %d, %d pixels of %d bytes %d apart: outside %d, same %d\n", offset, pixels, bytes, from,
           (int)outside, (int)same);
  }
}

// the generic filter gradient: additions of a lane, chunks of a grid, and the workspace of its sums
static void check_generic(const Conv& c) {
  const int64_t chunks = nhwc::generic_chunks(c), per = (nhwc::out_pixels(c) + chunks - 1) / chunks;
  const int64_t one = c.C * c.m * (c.kh * c.kw + 1) * 4;
  ++checks;
  const bool full = chunks == 4096 || (chunks + 1) * one > (int64_t(1) << 30);
  if ((per + 7) / 8 <= 1024 || full)
    if (chunks <= 4096 && nhwc::bwd_workspace_bytes(c) >= (size_t)(chunks * one)) return;
  ++fails;
  printf("FAIL generic N=%lld C=%lld H=%lld W=%lld k=%d: %lld chunks of %lld pixels, workspace %zu\n", (long long)c.N,
         (long long)c.C, (long long)c.H, (long long)c.W, c.kh, (long long)chunks, (long long)per, nhwc::bwd_workspace_bytes(c));
}

int main() {
  for (int64_t N : {1, 5, 64})
    for (int64_t C : {1, 40, 1024, 40000})
      for (int64_t side : {9, 31, 300, 3000})
        for (int k : {1, 4, 9, 31})
          if (side >= k) check_generic(mk(N, C, side, side + 1, k, 1, 0, DWCONV_F32));
  for (int i = 0; i < 4096; ++i) arena[i] = (uint8_t)(i * 37 + (i >> 8));
  for (int offset = 0; offset < 8; ++offset)
    for (int pixels : {1, 2, 7})
      for (int bytes = 1; bytes < 90; ++bytes)
        for (int gap : {0, 1, 6, 40}) check_reads(offset, pixels, bytes + gap, bytes);
  for (int s : {1, 2}) {
    check_rows(mk(1, 1 << 14, 2, 1 << 21, 3, s, 1, DWCONV_BF16), false);
    check_rows(mk(1, 1 << 14, 2, (1 << 21) - 1, 3, s, 1, DWCONV_BF16), true);
    check_rows(mk(1, 33, 2, 1 << 27, 3, s, 1, DWCONV_BF16), true);
  }
  for (int dtype : {DWCONV_F32, DWCONV_BF16})
    for (int k : {3, 5, 7})
      for (int s : {1, 2})
        for (int64_t N : {1, 3})
          for (int64_t C : {17, 33, 65, 130, 287})
            for (int64_t H : {9, 31, 500, 2000, 4100, 8300, 10000, 16500, 33000, 70000})
              for (int64_t W : {5, 32, 61, 200}) check_room(mk(N, C, H, W, k, s, k / 2, dtype));
  if (!tall) {
    ++fails;
    printf("FAIL no shape is staged from one source alone\n");
  }
  printf("%d checks, %d shapes staged from one source alone, fails: %d\n", checks, tall, fails);
  return fails != 0;
}
