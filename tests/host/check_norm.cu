// CPU check of the group norm's plans: additions that a thread chains, and the
// workspace against what each family lays out in it.
#include <cstdio>
#include "norm_slab.h"

namespace dwconv {
// what the planner's file calls in others; nothing here is launched
cudaError_t act8_encode(int64_t, int64_t, int64_t, int, const void*, const Act8&, cudaStream_t) { return cudaErrorNotSupported; }
namespace norm {
namespace slab {
#define X(T)                                                                                                            \
  template <>                                                                                                           \
  cudaError_t run_fwd<T>(const Norm&, const Plan&, bool, const T*, const T*, const T*, T*, float*, float*, const Act8&, \
                         const Sums&, cudaStream_t) {                                                                   \
    return cudaErrorNotSupported;                                                                                       \
  }                                                                                                                     \
  template <>                                                                                                           \
  cudaError_t run_bwd<T>(const Norm&, const Plan&, bool, const T*, const Act8&, const T*, const T*, const T*,           \
                         const float*, const float*, T*, const Sums&, cudaStream_t) {                                   \
    return cudaErrorNotSupported;                                                                                       \
  }
X(float) X(__half) X(__nv_bfloat16)
#undef X
}  // namespace slab
}  // namespace norm
}  // namespace dwconv
#include "norm.cu"

using namespace dwconv;
using norm::Norm;
static int fails = 0, checks = 0, streams = 0, splits = 0;

static Norm mk(int64_t N, int64_t P, int C, int G, int dtype) {
  Norm g{};
  g.N = N; g.P = P; g.C = C; g.G = G; g.D = C / G; g.dtype = dtype; g.eps = 1e-5f;
  g.xs = g.ys = C;
  return g;
}

// Rows that a thread adds up: at most this many, unless the chunks are as many as the kernels take.
constexpr int64_t kMost = 4096;

static void report(const char* what, const Norm& g, int V, int keep, int64_t a, int64_t b) {
  ++fails;
  if (fails <= 40)
    printf("FAIL %s: N=%lld P=%lld C=%d G=%d dtype=%d V=%d keep=%d: %lld of %lld\n", what, (long long)g.N, (long long)g.P,
           g.C, g.G, g.dtype, V, keep, (long long)a, (long long)b);
}

static void check(const Norm& g) {
  const int es = g.dtype == DWCONV_F32 ? 4 : 2;
  for (int pass = 0; pass < 2; ++pass) {
    const size_t size = norm::workspace_bytes(g, pass);
    for (int V : {8, 4, 0})  // 0: channels apart
      for (int source : {0, 32, 64, 128}) {  // forward: the checkpoint's block; backward: codes (any but 0)
        const bool strided = V == 0;
        if (V * es > 16 || (V && g.C % V) || (pass && source > 32)) continue;
        norm::slab::Plan k;
        const norm::Family f = norm::plan_family(g, strided ? 4 : V, strided, es, pass ? 0 : source,
                                                 pass ? (source ? 1 : es) : 0, &k);
        ++checks;
        size_t need;
        if (f == norm::kSplit) {
          if (!pass && source) continue;  // such a forward runs without the checkpoint
          const norm::Cut c = norm::plan_cut(g, V * es == 16 ? V : 1);
          const int64_t lane = (c.rows + c.rl - 1) / c.rl;
          if (lane > kMost && c.chunks < 256) report("rows of a split thread", g, V, source, lane, kMost);
          need = 8 * ((size_t)(g.N * g.G) + (size_t)g.N * c.chunks * (size_t)g.C);
          ++splits;
        } else {
          const int64_t lane = ((int64_t)k.rows + k.rl - 1) / k.rl;
          if (lane > kMost && k.parts < norm::slab::kMaxParts) report("rows of a thread", g, V, source, lane, kMost);
          const size_t parts = f == norm::kSlabs ? 1 : (size_t)k.parts;
          if ((int64_t)k.parts * k.rows < g.P || k.parts > norm::slab::kMaxParts) report("parts", g, V, source, k.parts, k.rows);
          const int smem = k.data_bytes + norm::slab::scratch_bytes(k, pass);
          if (smem > norm::slab::kMostSmem) report("shared memory", g, V, source, smem, norm::slab::kMostSmem);
          need = f == norm::kSlabs && !pass ? 0 : 8 * (size_t)g.N * parts * ((size_t)g.G + (pass ? (size_t)g.C : 0));
          streams += f == norm::kStream;
        }
        if (need > size) report("workspace", g, V, source, (int64_t)need, (int64_t)size);
      }
  }
}

int main() {
  for (int dtype : {DWCONV_F32, DWCONV_BF16})
    for (int64_t N : {1, 3, 40, 460, 512, 5000})
      for (int64_t P : {1, 49, 784, 12544, 66049, 262144, 1048576, 4194304, 30000000})
        for (int C : {1, 8, 20, 64, 96, 320, 1024, 1536, 2048, 2056, 4096, 6150})
          for (int G : {1, 2, 8, 32, 96})
            if (C % G == 0) check(mk(N, P, C, G, dtype));
  if (!streams || !splits) {
    ++fails;
    printf("FAIL families: %d streams, %d splits\n", streams, splits);
  }
  printf("%d checks, %d streams, %d splits, fails: %d\n", checks, streams, splits, fails);
  return fails != 0;
}
