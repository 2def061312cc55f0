// The host side of csrc/orthogonalize.hip (workspace layout, plans, launch sequence) under the sanitizers, for every
// path and many shapes: stand-ins of the HIP runtime take the launches and look at what they are given. Every buffer in
// the workspace has its whole extent, computed from what the kernel does, inside the workspace; no two buffers that one
// kernel reads and writes overlap; grids and workgroups are within the limits. Nothing is launched or dereferenced.
#include <stdio.h>
#include <string.h>

#include <functional>
#include <initializer_list>
#include <map>
#include <vector>

#include "orthogonalize.hip"

namespace {

long g_launches = 0, g_failures = 0;
const char* g_what = "";
#define CHECK(c)                                                                         \
  do {                                                                                   \
    if (!(c) && ++g_failures < 20) printf("%s:%d: %s (%s)\n", __FILE__, __LINE__, #c, g_what); \
  } while (0)

// a made-up address, near the end of what a size can be added to
char* const kWorkspace = reinterpret_cast<char*>(uintptr_t(0x6000000000000000));
size_t g_bytes = 0;

struct Extent {
  const char* from;
  size_t bytes;
};
Extent inside(const void* p, size_t bytes) {
  const char* c = static_cast<const char*>(p);
  CHECK(c >= kWorkspace && bytes <= g_bytes && c <= kWorkspace + (g_bytes - bytes));
  return {c, bytes};
}
void apart(const std::vector<Extent>& a, const std::vector<Extent>& b) {
  for (const Extent& x : a)
    for (const Extent& y : b) CHECK(x.from + x.bytes <= y.from || y.from + y.bytes <= x.from);
}

typedef std::function<void(dim3, void**)> Look;
std::map<const void*, Look> g_kernels;
template <class T>
const T& arg(void** args, int i) {
  return *static_cast<const T*>(args[i]);
}

template <class G, bool SYM>
struct Product {
  static std::vector<Extent> operand(const ProductArgs& a, const Operands& o) {
    const size_t all = (size_t)a.E * (size_t)o.mat * 2;
    CHECK(G::TERMS == 1 || o.plane * 2 == (int64_t)all);
    return {inside(o.at, all * G::TERMS)};
  }
  static std::vector<Extent> sums(const ProductArgs& a) {
    if (a.parts <= 1) return {};
    CHECK(a.parts <= kMaxParts && a.parts <= a.K / (kStages * G::BK));
    return {inside(a.sums, (size_t)kXcds * a.rest * a.parts * G::BM * G::BM * 4)};
  }
  // what the epilogue reads and writes
  static void out(const ProductArgs& a, bool last, std::vector<Extent>& reads, std::vector<Extent>& writes, bool c) {
    if (last) return;
    const size_t all = (size_t)a.E * a.rows * a.cols * 2;
    CHECK(G::TERMS == 1 || a.d_plane * 2 == (int64_t)all);
    writes.push_back(inside(a.d, all * G::TERMS));
    if (c) reads.push_back(operand(a, a.c)[0]);
  }
  static void common(const ProductArgs& a) {
    CHECK(a.E >= 1 && a.K > 0 && a.K % kPad == 0 && a.rows % kPad == 0 && a.cols % kPad == 0);
    CHECK((G::A::KS ? a.K : a.rows) == a.a.rows && (G::B::KS ? a.K : a.cols) == a.b.rows);
    CHECK(a.a.mat == a.K * a.rows && a.b.mat == a.K * a.cols);
    CHECK(!SYM || a.rows == a.cols);
    if (a.power) inside(a.first, (size_t)a.E * 4);
  }
  template <int KIND>
  static void look(bool join, dim3 grid, void** args) {
    const ProductArgs& a = arg<ProductArgs>(args, 0);
    common(a);
    const int64_t tiles = tiles_of(a, G::BM, SYM), each = (tiles + kXcds - 1) / kXcds;
    std::vector<Extent> reads, writes;
    if (join) {
      CHECK(a.parts > 1 && a.rest >= each && grid.x == (unsigned)(a.rest * kXcds * 4 * Passes<G>::ALL));
      reads = sums(a);
    } else {
      reads = {operand(a, a.a)[0], operand(a, a.b)[0]};
      CHECK(grid.x % kXcds == 0 && grid.x / kXcds >= 1 && grid.x / kXcds <= (unsigned)G::SLOTS);
      CHECK(a.parts > 1 || grid.x / kXcds >= (unsigned)(each < G::SLOTS ? each : G::SLOTS));
    }
    if (join || a.parts <= 1) out(a, KIND >= kLast, reads, writes, KIND == kPolynomial);
    else writes = sums(a);
    apart(reads, writes);
  }
  template <int KIND, typename TO>
  static void add() {
    g_kernels[reinterpret_cast<const void*>(&product_kernel<G, SYM, KIND, TO>)] = [](dim3 g, void** p) { look<KIND>(false, g, p); };
    g_kernels[reinterpret_cast<const void*>(&join_kernel<G, SYM, KIND, TO>)] = [](dim3 g, void** p) { look<KIND>(true, g, p); };
  }
};

template <int TERMS, typename TI>
void add_products() {
  Product<Big<true, true, TERMS>, true>::template add<kProduct, f16>();
  Product<Small<true, true, TERMS>, true>::template add<kProduct, f16>();
  Product<Big<false, false, TERMS>, true>::template add<kProduct, f16>();
  Product<Small<false, false, TERMS>, true>::template add<kProduct, f16>();
  Product<Big<false, false, TERMS>, true>::template add<kPolynomial, f16>();
  Product<Small<false, false, TERMS>, true>::template add<kPolynomial, f16>();
  Product<Big<false, false, TERMS>, false>::template add<kProduct, f16>();
  Product<Small<false, false, TERMS>, false>::template add<kProduct, f16>();
  Product<Big<false, true, TERMS>, false>::template add<kProduct, f16>();
  Product<Small<false, true, TERMS>, false>::template add<kProduct, f16>();
  Product<Big<false, false, TERMS>, false>::template add<kLast, TI>();
  Product<Small<false, false, TERMS>, false>::template add<kLast, TI>();
  Product<Big<false, true, TERMS>, false>::template add<kLast, TI>();
  Product<Small<false, true, TERMS>, false>::template add<kLast, TI>();
  Product<Big<false, false, TERMS>, false>::template add<kUpdate, TI>();
  Product<Small<false, false, TERMS>, false>::template add<kUpdate, TI>();
  Product<Big<false, true, TERMS>, false>::template add<kUpdate, TI>();
  Product<Small<false, true, TERMS>, false>::template add<kUpdate, TI>();
}

template <typename TI, int TERMS>
void add_scale() {
  g_kernels[reinterpret_cast<const void*>(&scale_kernel<TI, TERMS>)] = [](dim3 grid, void** p) {
    const OrthArgs& a = arg<OrthArgs>(p, 0);
    const int blocks = arg<int>(p, 3);
    const int64_t rows = arg<int64_t>(p, 7), cols = arg<int64_t>(p, 8), plane = arg<int64_t>(p, 9);
    const size_t all = (size_t)a.E * rows * cols * 2;
    CHECK(blocks >= 1 && blocks <= 256 && grid.y == (unsigned)a.E && rows >= a.m && cols >= a.n && rows * (cols / 8) < (int64_t(1) << 32));
    CHECK(TERMS == 1 || plane * 2 == (int64_t)all);
    std::vector<Extent> writes{inside(arg<f16*>(p, 5), all * TERMS), inside(arg<float*>(p, 10), (size_t)a.E * 4)};
    if (f16* const frags = arg<f16*>(p, 6)) {
      writes.push_back(inside(frags, all * TERMS));
      apart({writes[0]}, {writes[2]});
    }
    apart({inside(arg<const double*>(p, 2), (size_t)a.E * blocks * 8)}, writes);
  };
}

template <typename TI>
void add_type() {
  g_kernels[reinterpret_cast<const void*>(&square_kernel<TI>)] = [](dim3 grid, void** p) {
    CHECK(grid.x >= 1 && grid.x <= 256 && grid.y == (unsigned)arg<OrthArgs>(p, 0).E);
    inside(arg<double*>(p, 2), (size_t)grid.x * grid.y * 8);
  };
  add_scale<TI, 2>();
  g_kernels[reinterpret_cast<const void*>(&scale_turned_kernel<TI>)] = [](dim3 grid, void** p) {
    const OrthArgs& a = arg<OrthArgs>(p, 0);
    const int64_t rows = arg<int64_t>(p, 7);
    const size_t all = (size_t)a.E * rows * kStrip * 2;
    CHECK(arg<int64_t>(p, 8) * 2 == (int64_t)all && grid.x == (unsigned)(kStrip / 32 * (rows / 64)) && rows >= a.n && a.m <= kStrip);
    const Extent x = inside(arg<f16*>(p, 5), all * 2), f = inside(arg<f16*>(p, 6), all * 2);
    apart({x}, {f});
    apart({inside(arg<const double*>(p, 2), (size_t)a.E * arg<int>(p, 3) * 8)}, {x, f, inside(arg<float*>(p, 9), (size_t)a.E * 4)});
  };
  auto strip = [](bool last, dim3 grid, void** p) {
    const OrthArgs& a = arg<OrthArgs>(p, 0);
    const StripArgs& t = arg<StripArgs>(p, 1);
    const size_t x = (size_t)a.E * t.rows * kStrip * 2, sq = (size_t)a.E * kStrip * kStrip * 2;
    CHECK(t.rows % kStripLong == 0 && t.x_plane * 2 == (int64_t)x && t.a_plane * 2 == (int64_t)sq);
    CHECK(grid.x >= (unsigned)(a.E * (t.rows / kStripLong) * (kStrip / kStripRows)) && grid.x % (kXcds * (kStrip / kStripRows)) == 0);
    const std::vector<Extent> reads{inside(t.A, sq * 2), inside(t.x, x * 2), inside(t.first, (size_t)a.E * 4)};
    if (!last) apart(reads, {inside(t.to, x * 2), inside(t.panels, x * 2)});
  };
  g_kernels[reinterpret_cast<const void*>(&strip_kernel<TI, true>)] = [strip](dim3 g, void** p) { strip(true, g, p); };
  g_kernels[reinterpret_cast<const void*>(&strip_kernel<TI, false>)] = [strip](dim3 g, void** p) { strip(false, g, p); };
  g_kernels[reinterpret_cast<const void*>(&small_kernel<TI>)] = [](dim3 grid, void** p) {
    const OrthArgs& a = arg<OrthArgs>(p, 0);
    CHECK(grid.x == (unsigned)a.E && (a.m <= kSmallSide || a.n <= kSmallSide) && long_side(a) <= kSmallLong);
  };
  auto thin = [](dim3 grid, void** p) {
    const OrthArgs& a = arg<OrthArgs>(p, 0);
    const ThinArgs& t = arg<ThinArgs>(p, 1);
    const size_t groups = (size_t)grid.x * grid.y;
    CHECK(grid.y == (unsigned)a.E && t.each % 128 == 0 && t.each <= kSmallLong && (int64_t)grid.x * t.each >= long_side(a));
    CHECK((int64_t)(grid.x - 1) * t.each < long_side(a) && t.blocks <= 256);
    const std::vector<Extent> all{inside(t.partial, (size_t)a.E * t.blocks * 8), inside(t.first, (size_t)a.E * 4),
                                  inside(t.x, groups * 4 * kSmallSide * kSmallLong), inside(t.P, (size_t)a.E * 4 * kSmallSide * kSmallSide),
                                  inside(t.parts, groups * 4 * kSmallSide * kSmallSide)};
    for (size_t i = 0; i < all.size(); ++i)
      for (size_t j = 0; j < i; ++j) apart({all[i]}, {all[j]});
  };
  g_kernels[reinterpret_cast<const void*>(&thin_kernel<TI, true, false>)] = thin;
  g_kernels[reinterpret_cast<const void*>(&thin_kernel<TI, false, true>)] = thin;
  g_kernels[reinterpret_cast<const void*>(&thin_kernel<TI, false, false>)] = thin;
}

void add_kernels() {
  add_type<bf16>();
  add_type<float>();
  add_scale<bf16, 1>();
  add_products<1, bf16>();
  add_products<2, bf16>();
  add_products<2, float>();
  Product<Big<true, true, 2>, true>::add<kFragments, f16>();
  Product<Small<true, true, 2>, true>::add<kFragments, f16>();
  g_kernels[reinterpret_cast<const void*>(&polynomial_kernel)] = [](dim3 grid, void** p) {
    const size_t sq = (size_t)grid.x * kPad * kPad * 2;
    CHECK(grid.x == (unsigned)arg<OrthArgs>(p, 0).E && arg<int64_t>(p, 4) * 2 == (int64_t)sq);
    apart({inside(arg<const f16*>(p, 2), sq * 2)}, {inside(arg<f16*>(p, 3), sq * 2)});
  };
  g_kernels[reinterpret_cast<const void*>(&thin_polynomial_kernel)] = [](dim3 grid, void** p) {
    const size_t parts = (size_t)arg<int>(p, 2);
    apart({inside(arg<ThinArgs>(p, 1).parts, grid.x * parts * 4 * kSmallSide * kSmallSide)},
          {inside(arg<char*>(p, 4), (size_t)grid.x * 4 * kSmallSide * kSmallSide)});
  };
}

struct Launch {
  dim3 grid, block;
  size_t shared;
  hipStream_t stream;
} g_launch;

}  // namespace

// ---- the HIP runtime's part --------------------------------------------------------------
extern "C" {
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t shared, hipStream_t stream) {
  g_launch = {grid, block, shared, stream};
  return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* shared, hipStream_t* stream) {
  *grid = g_launch.grid;
  *block = g_launch.block;
  *shared = g_launch.shared;
  *stream = g_launch.stream;
  return hipSuccess;
}
hipError_t hipLaunchKernel(const void* f, dim3 grid, dim3 block, void** args, size_t, hipStream_t) {
  ++g_launches;
  CHECK(grid.x >= 1 && grid.y >= 1 && grid.z == 1 && grid.y <= 65535 && block.y == 1 && block.z == 1);
  CHECK(block.x >= 64 && block.x <= 1024 && (uint64_t)grid.x * block.x < (uint64_t(1) << 32));
  const auto k = g_kernels.find(f);
  CHECK(k != g_kernels.end());
  if (k != g_kernels.end()) k->second(grid, args);
  return hipSuccess;
}
hipError_t hipGetLastError() { return hipSuccess; }
// (registration of the kernels, of which there is no device code here)
void** __hipRegisterFatBinary(const void*) {
  static void* none = nullptr;
  return &none;
}
void __hipRegisterFunction(void**, const void*, char*, const char*, unsigned, void*, void*, void*, void*, int*) {}
void __hipUnregisterFatBinary(void**) {}
}

int main() {
  add_kernels();
  const int64_t sides[] = {1, 9, 24, 25, 64, 65, 128, 129, 200, 256, 257, 384, 385, 512, 520, 1000, 1408, 2048, 4096, 12288, 12289, 14336, 16384, 1 << 18};
  static char text[200];
  g_what = text;
  long cases = 0, terms[3] = {}, strips = 0, parts = 0;
  for (int64_t m : sides)
    for (int64_t n : sides) {
      if (m > 16384 && n > 16384) continue;
      for (int E : {1, 2, 5, 16, 64})
        for (int type : {0, 1})
          for (int steps : {1, 2, 3, 5, 6})
            for (int update : {0, 1}) {
              OrthArgs a{};
              a.m = m;
              a.n = n;
              a.E = E;
              a.bf16 = type;
              a.steps = steps;
              a.a = 3.4445f;
              a.b = -4.7750f;
              a.c = 2.0315f;
              a.eps = 1e-7f;
              a.g = a.out = reinterpret_cast<void*>(0x10000);
              a.momentum = update ? reinterpret_cast<float*>(0x20000) : nullptr;
              a.ws = kWorkspace;
              snprintf(text, sizeof(text), "%d of %ld x %ld, type %d, %d steps, update %d", E, (long)m, (long)n, type, steps, update);
              g_bytes = orthogonalize_workspace(a);
              CHECK(g_bytes >= 256 && g_bytes % 256 == 0);
              const long before = g_launches;
              CHECK(launch_orthogonalize(a, nullptr) == hipSuccess);
              CHECK(g_launches > before);
              ++cases;
              ++terms[terms_of(a)];
              strips += is_strip(a);
              const Layout l = layout_of(a);
              parts += !is_small(a) && !is_thin(a) && l.x[0] > l.sums;
            }
    }
  CHECK(terms[1] && terms[2] && strips && parts);
  printf("%ld cases (%ld in one term, %ld in two, %ld in strips, %ld with parts), %ld launches, passed: %ld failure(s)\n", cases, terms[1],
         terms[2], strips, parts, g_launches, g_failures);
  return g_failures != 0;
}
