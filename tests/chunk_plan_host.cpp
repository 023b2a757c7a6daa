// The plan of attention of new tokens run on the CPU: the library's own host checks and plan header, a wave as 64 fibers that
// meet at each operation between lanes.  plan_of() gives what every workgroup would walk and what the join would read.
#include <ucontext.h>

#include <algorithm>
#include <cstdlib>
#include <vector>

#include "attn/fq_attn.h"
#include "attn/fq_host_util.h"

// ---- a wave ------------------------------------------------------------------------------
namespace {

constexpr int kLanes = 64;
ucontext_t g_lane[kLanes], g_main;
char* g_stack[kLanes];
int g_now, g_slot[2][kLanes], g_op[kLanes];
struct Index {
  int x;
} threadIdx, blockIdx;

// Every lane's v at the same operation: a lane goes on once all have come there.
const int* meet(int v) {
  const int me = g_now, at = g_op[me]++ & 1;
  g_slot[at][me] = v;
  g_now = (me + 1) % kLanes;
  threadIdx.x = g_now;
  swapcontext(&g_lane[me], &g_lane[g_now]);
  return g_slot[at];
}
int read_lane(int v, int w) {
  const int* const all = meet(v);
  return w < 0 || w >= kLanes ? (std::abort(), 0) : all[w];
}
int scan(int v) {
  const int me = g_now;
  const int* const all = meet(v);
  unsigned sum = 0;
  for (int i = 0; i <= me; ++i) sum += static_cast<unsigned>(all[i]);
  return static_cast<int>(sum);
}
uint64_t ballot(bool v) {
  const int* const all = meet(v);
  uint64_t m = 0;
  for (int i = 0; i < kLanes; ++i) m |= static_cast<uint64_t>(all[i] != 0) << i;
  return m;
}

}  // namespace

#define __builtin_amdgcn_readlane read_lane
#define __ballot ballot
#define wave_scan scan
#ifndef __forceinline__
#define __forceinline__ inline
#endif
using std::max;
using std::min;
#include "attn/fq_attn_chunk_plan.h"

// ---- the library around it ---------------------------------------------------------------------
namespace fq {

bool is_contiguous(const fq_tensor&) { return true; }
bool strides_ok(const fq_tensor&) { return true; }
bool shape_is(const fq_tensor& t, int nd, int64_t a, int64_t b, int64_t c) {
  const int64_t s[3] = {a, b, c};
  bool ok = t.ndim == nd;
  for (int d = 0; ok && d < nd; ++d) ok = t.shape[d] == s[d];
  return ok;
}
void clear_last_error() {}
fq_status fail_runtime(const char*, hipError_t) { return FQ_ERR_RUNTIME; }
bool device_is_gfx950() { return true; }
ChunkArgs g_args;
hipError_t launch_attn_chunk_16(const ChunkArgs& a, void*, hipStream_t) { return g_args = a, hipSuccess; }
hipError_t launch_attn_chunk_int8(const ChunkArgs& a, void*, hipStream_t) { return g_args = a, hipSuccess; }
hipError_t launch_attn_chunk_e4m3(const ChunkArgs& a, void*, hipStream_t) { return g_args = a, hipSuccess; }
hipError_t launch_attn_chunk_int4(const ChunkArgs& a, void*, hipStream_t) { return g_args = a, hipSuccess; }
hipError_t launch_attn_chunk_fp4(const ChunkArgs& a, void*, hipStream_t) { return g_args = a, hipSuccess; }

}  // namespace fq

namespace {

using namespace fq;

// One segment that a workgroup walks a part of, or (joined) one whose parts the second launch joins.
struct Record {
  int joined, run, b, head, tile, q0, row0, row1, off, lk, n, sinks, lo, u0, u1, whole, part, parts;
};
std::vector<Record> g_records;
size_t g_most;

void put(int joined, int run, const Segment& sg, const Walk& wk, int u0, int u1, bool whole, int parts) {
  if (g_now == 0)
    g_records.push_back(Record{joined, run, sg.b, sg.head, sg.tile, sg.s.q0, wk.row0, wk.row1, sg.s.off, sg.s.lk, wk.n, wk.sinks, wk.lo, u0, u1, whole,
                               part_at(run, u0), parts});
  if (g_records.size() > g_most) std::abort();
}

void walk_block() {
  const Run run = run_of(g_args);
  if (run.last <= run.first) return;
  Segment sg = segment_at(g_args, run.first);
  if (sg.s.tiles == 0) return;
  do {
    const Walk wk = walk_of(g_args, sg.s, sg.tile);
    const Share sh = share_of(g_args, run, sg, wk);
    if (!sh.whole && sh.u0 >= sh.u1) continue;
    put(0, run.i, sg, wk, sh.u0, sh.u1, sh.whole, 0);
  } while (next_segment(g_args, run, sg));
}
void join_block() {
  const Shared sh = shared_from(g_args, blockIdx.x);
  if (sh.parts) put(1, blockIdx.x, sh.sg, sh.wk, 0, sh.wk.n, false, sh.parts);
}

void (*g_block)();
void lane_main() {
  g_block();
  // (all lanes end at the same place, one after the other)
  const int me = g_now;
  g_now = me + 1 < kLanes ? me + 1 : 0;
  threadIdx.x = g_now;
  setcontext(me + 1 < kLanes ? &g_lane[me + 1] : &g_main);
}
void run_block(int index, void (*block)()) {
  constexpr size_t kStack = 1 << 16;
  blockIdx.x = index;
  g_block = block;
  g_now = threadIdx.x = 0;
  for (int i = 0; i < kLanes; ++i) {
    if (!g_stack[i]) g_stack[i] = static_cast<char*>(std::malloc(kStack));
    g_op[i] = 0;
    getcontext(&g_lane[i]);
    g_lane[i].uc_stack.ss_sp = g_stack[i];
    g_lane[i].uc_stack.ss_size = kStack;
    g_lane[i].uc_link = nullptr;
    makecontext(&g_lane[i], lane_main, 0);
  }
  swapcontext(&g_main, &g_lane[0]);
}

}  // namespace

// sizes: Tq, B, Hq, Hkv, D, page size, table width, window, sinks.  Returns the number of records (in `out`, of at most `most`), or minus the status
// of the call; args: tile_rows, tokens, tile_heads, head_tiles, heads, runs, single, and how many parts the workspace has.
extern "C" int64_t plan_of(const int32_t* sizes, const int32_t* cu, const int32_t* lengths, int32_t* args, int32_t* out, int64_t most) {
  const int64_t Tq = sizes[0], B = sizes[1], Hq = sizes[2], Hkv = sizes[3], D = sizes[4], P = sizes[5], W = sizes[6];
  void* const dummy = reinterpret_cast<void*>(uintptr_t(1) << 20);
  auto tens = [&](int32_t dt, std::initializer_list<int64_t> shape, const void* data) {
    fq_tensor t{};
    t.data = const_cast<void*>(data);
    t.dtype = dt;
    t.ndim = static_cast<int32_t>(shape.size());
    int64_t step = 1;
    std::copy(shape.begin(), shape.end(), t.shape);
    for (int d = t.ndim - 1; d >= 0; step *= t.shape[d--]) t.strides[d] = step;
    return t;
  };
  const fq_tensor q = tens(FQ_DT_BFLOAT16, {Tq, Hq, D}, dummy), kc = tens(FQ_DT_BFLOAT16, {4, Hkv, P, D}, dummy), bt = tens(FQ_DT_INT32, {B, W}, dummy),
                  c = tens(FQ_DT_INT32, {B + 1}, cu), n = tens(FQ_DT_INT32, {B}, lengths);
  uint64_t size = 0;
  fq_status st = fq_attn_chunk_get_workspace_size(&q, &kc, &bt, &c, sizes[7], sizes[8], &size);
  if (st == FQ_SUCCESS)
    st = fq_attn_chunk(&q, &kc, nullptr, &kc, nullptr, &bt, &c, &n, sizes[7], sizes[8], 0.0, &q, nullptr, dummy, size, nullptr);
  if (st != FQ_SUCCESS) return -static_cast<int64_t>(st);
  const int64_t padded = D <= 64 ? 64 : D <= 128 ? 128 : 256;
  const int32_t a[8] = {g_args.tile_rows, g_args.tokens, g_args.tile_heads, g_args.head_tiles, g_args.heads, g_args.runs, g_args.single,
                        static_cast<int32_t>(size / ((padded + 2) * g_args.tile_rows * 4))};
  std::copy(a, a + 8, args);
  g_records.clear();
  g_most = static_cast<size_t>(most);
  for (int i = 0; i < 8 * ((g_args.runs + 7) / 8); ++i) run_block(i, walk_block);
  if (!g_args.single)
    for (int i = 0; i + 1 < g_args.runs; ++i) run_block(i, join_block);
  std::copy(g_records.begin(), g_records.end(), reinterpret_cast<Record*>(out));
  return static_cast<int64_t>(g_records.size());
}
