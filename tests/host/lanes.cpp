// Runs a kernel's workgroups on the host, one after another.  Every lane is a fibre
// with a stack of its own; a wave's lanes run on until they wait for each other (a
// collective operation) or for the workgroup (a barrier), and which wave goes on next
// is drawn at random.  Ends the program where lanes wait for what never comes, meet in
// different collectives, or leave loads in flight.
#include <hip/hip_runtime.h>
#include <stdio.h>
#include <stdlib.h>
#include <sys/mman.h>

#include <random>

namespace lanes {

Index block, grid;

// Saves the running fibre's registers on its stack and its stack pointer in *save,
// and goes on with the fibre whose stack pointer is `to` (x86-64, System V).
extern "C" void lanes_switch(void** save, void* to);
asm(R"(
.text
.globl lanes_switch
lanes_switch:
  pushq %rbp
  pushq %rbx
  pushq %r12
  pushq %r13
  pushq %r14
  pushq %r15
  movq %rsp, (%rdi)
  movq %rsi, %rsp
  popq %r15
  popq %r14
  popq %r13
  popq %r12
  popq %rbx
  popq %rbp
  ret
)");

namespace {

constexpr size_t kStack = 512 << 10;
constexpr size_t kValue = 64;  // bytes of an exchanged value

struct Load {  // a direct load in flight
  void* dst;
  uint8_t n, bytes[16];
};

enum Wait { kReady, kWave, kBarrier };

struct Fibre {
  void* sp;
  bool done;
  Wait wait;
  std::vector<Load> loads;
};

// Values of an exchange; two sets in turn, since a lane may still read one while
// another lane is in the next.
struct Wave {
  int running, arrived, turn;
  size_t size;
  uint64_t came, gave[2];
  uint8_t values[2][64 * kValue];
};

std::vector<Fibre> fibres;
std::vector<Wave> waves;
std::vector<uint8_t*> stacks;
int cur, running, at_barrier;
void* main_sp;
const std::function<void()>* body;
uint8_t* lds_at;
size_t lds_size;
bool late = true;
std::mt19937 rng(1);

int first_of(int w) { return w * 64; }
int end_of(int w) { return std::min<int>(w * 64 + 64, (int)fibres.size()); }
bool ready(int i) { return !fibres[i].done && fibres[i].wait == kReady; }

// Another lane of this wave if one can run, else a lane of some other wave.
void next() {
  const int self = cur, w = cur >> 6;
  int to = -1;
  for (int k = 1; k < 64 && to < 0; ++k) {
    const int i = first_of(w) + (cur - first_of(w) + k) % 64;
    if (i < end_of(w) && ready(i)) to = i;
  }
  const int nw = (int)waves.size(), start = rng() % nw;
  for (int k = 0; k < nw && to < 0; ++k) {
    const int v = (start + k) % nw;
    for (int i = first_of(v); i < end_of(v) && to < 0; ++i)
      if (ready(i)) to = i;
  }
  if (to < 0 && running > 0) fail("lanes wait for what never comes");
  if (to == self) return;
  if (to >= 0) cur = to;
  lanes_switch(&fibres[self].sp, to < 0 ? main_sp : fibres[to].sp);
}

void complete_exchange(int w) {
  Wave& v = waves[w];
  v.gave[v.turn] = v.came;
  v.arrived = 0;
  v.turn ^= 1;
  for (int i = first_of(w); i < end_of(w); ++i)
    if (fibres[i].wait == kWave) fibres[i].wait = kReady;
}

void complete_barrier() {
  if (running == 0 || at_barrier < running) return;
  at_barrier = 0;
  for (Fibre& f : fibres)
    if (f.wait == kBarrier) f.wait = kReady;
}

void lane_main() {
  (*body)();
  Fibre& f = fibres[cur];
  if (!f.loads.empty()) fail("a lane ends with loads in flight");
  f.done = true;
  --running;
  const int w = cur >> 6;
  --waves[w].running;
  // what the others wait for may have been this lane
  if (waves[w].running > 0 && waves[w].arrived == waves[w].running) complete_exchange(w);
  complete_barrier();
  next();
  fail("a finished lane ran");
}

}  // namespace

// late_loads: direct loads land when a wait asks for them, and until then neither the
// old bytes nor the new ones are there; else at once.
extern "C" void lanes_mode(int late_loads, int seed) {
  late = late_loads != 0;
  rng.seed(seed);
}

void fail(const char* what) {
  fprintf(stderr, "host run: %s (workgroup %u, thread %d)\n", what, block.x, cur);
  fflush(stderr);
  abort();
}

Index thread() { return {(unsigned)cur, 0, 0}; }
int lane() { return cur & 63; }
uint8_t* dynamic_lds() { return lds_at; }

const uint8_t* exchange(const void* value, size_t size, uint64_t* gave) {
  const int w = cur >> 6;
  Wave& v = waves[w];
  if (size > kValue) fail("an exchanged value is too large");
  if (v.arrived == 0) {
    v.size = size;
    v.came = 0;
  } else if (v.size != size) {
    fail("lanes of a wave meet in different operations");
  }
  const int turn = v.turn;
  memcpy(v.values[turn] + lane() * size, value, size);
  v.came |= 1ull << lane();
  if (++v.arrived == v.running) {
    complete_exchange(w);
  } else {
    fibres[cur].wait = kWave;
    while (fibres[cur].wait != kReady) next();
  }
  *gave = v.gave[turn];
  return v.values[turn];
}

void barrier() {
  ++at_barrier;
  fibres[cur].wait = kBarrier;
  complete_barrier();
  while (fibres[cur].wait != kReady) next();
}

void land(void* dst, const void* src, size_t n) {
  uint8_t* d = (uint8_t*)dst;
  if (d < lds_at || d + n > lds_at + lds_size) fail("a direct load outside the LDS");
  if (!late) {
    memcpy(dst, src, n);
    return;
  }
  Load l{dst, (uint8_t)n, {}};
  memcpy(l.bytes, src, n);
  fibres[cur].loads.push_back(l);
  memset(dst, 0xFB, n);
}

void wait_loads(int left) {
  std::vector<Load>& q = fibres[cur].loads;
  size_t k = 0;
  for (; q.size() - k > (size_t)left; ++k) memcpy(q[k].dst, q[k].bytes, q[k].n);
  q.erase(q.begin(), q.begin() + k);
}

void run(unsigned workgroups, unsigned threads, size_t lds, const std::function<void()>& kernel) {
  if (threads == 0 || threads > 1024 || lds > 160 * 1024) fail("the launch's shape");
  if (workgroups == 0 || (uint64_t)workgroups * threads > 0xFFFFFFFFull) fail("the launch's grid");
  while (stacks.size() < threads)
    stacks.push_back((uint8_t*)mmap(nullptr, kStack, PROT_READ | PROT_WRITE,
                                    MAP_PRIVATE | MAP_ANONYMOUS | MAP_NORESERVE, -1, 0));
  body = &kernel;
  grid = {workgroups, 1, 1};
  lds_size = lds;
  lds_at = (uint8_t*)aligned_alloc(16, lds / 16 * 16 + 16);
  fibres.resize(threads);
  waves.resize((threads + 63) / 64);
  for (unsigned b = 0; b < workgroups; ++b) {
    block = {b, 0, 0};
    memset(lds_at, 0xFD, lds);
    running = (int)threads;
    at_barrier = 0;
    for (size_t w = 0; w < waves.size(); ++w) {
      waves[w].arrived = waves[w].turn = 0;
      waves[w].running = end_of((int)w) - first_of((int)w);
    }
    for (unsigned i = 0; i < threads; ++i) {
      Fibre& f = fibres[i];
      f.done = false;
      f.wait = kReady;
      f.loads.clear();
      // a stack from which lanes_switch returns into lane_main
      void** sp = (void**)(stacks[i] + kStack - 64);
      *--sp = nullptr;
      *--sp = (void*)lane_main;
      for (int k = 0; k < 6; ++k) *--sp = nullptr;
      f.sp = sp;
    }
    cur = (int)(rng() % waves.size()) * 64;
    lanes_switch(&main_sp, fibres[cur].sp);
  }
  free(lds_at);
}

// ---- arithmetic -------------------------------------------------------------

float e4m3(uint32_t b) {
  const int e = b >> 3 & 15, m = b & 7;
  float v = e ? ldexpf((float)(8 + m), e - 10) : ldexpf((float)m, -9);
  if (e == 15 && m == 7) v = NAN;
  return b & 128 ? -v : v;
}

// Nearest of 4 significant bits (steps of 2^-9 below 2^-6), ties to even.
uint8_t to_e4m3(float v) {
  const uint8_t sign = signbit(v) ? 128 : 0;
  const float a = fabsf(v);
  if (!(a <= 464.f)) return sign | 0x7F;
  int e;
  frexpf(a, &e);
  const double step = ldexp(1.0, std::max(e - 1, -6) - 3), r = nearbyint(a / step) * step;
  if (r == 0) return sign;
  if (r > 448) return sign | 0x7F;
  frexp(r, &e);
  const int ex = std::max(e - 1, -6), q = (int)ldexp(r, 3 - ex);
  return sign | (q < 8 ? q : ((ex + 7) << 3) | (q - 8));
}

static float result(double sum) { return (float)sum; }
static float result(float sum) { return sum; }
static int result(int64_t sum) {
  if (sum != (int32_t)sum) fail("a 32-bit sum overflows");
  return (int)sum;
}

// The matrix instructions' layout: lane L gives elements of row (column) L % 16 of the
// operands, those of its group L / 16, and receives rows 4 (L / 16) + 0..3 of column
// L % 16.  add(sum, x, y): adds the products of two lanes' operands.
template <typename A, typename C, typename Sum, typename Add>
static C matrix(const A& a, const A& b, C c, Add add) {
  struct {
    A a, b;
  } v{a, b};
  uint64_t gave;
  const uint8_t* all = exchange(&v, sizeof(v), &gave);
  if (gave != ~0ull) fail("a matrix instruction of a part of a wave");
  for (int r = 0; r < 4; ++r) {
    Sum sum = c[r];
    for (int g = 0; g < 4; ++g)
      add(sum, all + (16 * g + 4 * (lane() >> 4) + r) * sizeof(v), all + (16 * g + (lane() & 15)) * sizeof(v) + sizeof(A));
    c[r] = result(sum);
  }
  return c;
}

f4 mfma_fp8(i8 a, i8 b, f4 c, int, int, int, int, int, int) {
  static const std::vector<double> value = [] {
    std::vector<double> t(256);
    for (int i = 0; i < 256; ++i) t[i] = e4m3(i);
    return t;
  }();
  return matrix<i8, f4, double>(a, b, c, [](double& sum, const uint8_t* x, const uint8_t* y) {
    for (int k = 0; k < 32; ++k) sum += value[x[k]] * value[y[k]];
  });
}

f4 mfma_f16(h8 a, h8 b, f4 c, int, int, int) {
  return matrix<h8, f4, float>(a, b, c, [](float& sum, const uint8_t* x, const uint8_t* y) {
    for (int k = 0; k < 8; ++k) sum += (float)((const _Float16*)x)[k] * (float)((const _Float16*)y)[k];
  });
}

i4 mfma_i8(i4 a, i4 b, i4 c, int, int, int) {
  return matrix<i4, i4, int64_t>(a, b, c, [](int64_t& sum, const uint8_t* x, const uint8_t* y) {
    for (int k = 0; k < 16; ++k) sum += (int)(int8_t)x[k] * (int)(int8_t)y[k];
  });
}

}  // namespace lanes
