// The library's scratch buffers over the fake CUDA runtime of host_lane_fake_cuda.cpp
// (CPU, no GPU): whose a buffer is.  That file's fakes are taken as they are; this one
// adds stream ids, which a handle alone does not give: cudaStreamPerThread is a stream
// in every host thread, and a destroyed stream's handle comes back for a new one.
//
// tests/test_shared_host.py compiles it with pad_api.cpp and pad_shared_api.cpp.
// Arguments: a scenario's name, and "no-ids" for a driver without cuStreamGetId.
#include <cuda.h>
#include <cuda_runtime.h>

#define cudaGetDriverEntryPoint fake_lane_entry_point
#define main fake_lane_main
#include "host_lane_fake_cuda.cpp"
#undef main
#undef cudaGetDriverEntryPoint

#include <algorithm>
#include <atomic>
#include <chrono>
#include <condition_variable>
#include <map>
#include <mutex>
#include <thread>

#include "pad_shared.h"

static bool no_ids = false;
static int ids_asked = 0;
static std::mutex ids_mu;
static std::map<cudaStream_t, unsigned long long> stream_ids;  // a reused handle gets another

static CUresult fake_stream_id(CUstream s, unsigned long long *id) {
  static std::atomic<unsigned long long> threads{1000000};
  static thread_local unsigned long long mine = ++threads;
  std::lock_guard<std::mutex> lock(ids_mu);
  ++ids_asked;
  *id = s == cudaStreamPerThread ? mine : stream_ids.count(s) ? stream_ids[s] : 1 + (unsigned long long)(uintptr_t)s;
  return CUDA_SUCCESS;
}
// (the lane's encoder records what it is asked for: one thread at a time)
static CUresult locked_encode(CUtensorMap *map, CUtensorMapDataType dt, cuuint32_t rank, void *addr,
                              const cuuint64_t *dims, const cuuint64_t *strides, const cuuint32_t *box,
                              const cuuint32_t *elem, CUtensorMapInterleave il, CUtensorMapSwizzle sw,
                              CUtensorMapL2promotion l2, CUtensorMapFloatOOBfill oob) {
  static std::mutex mu;
  std::lock_guard<std::mutex> lock(mu);
  return fake_encode(map, dt, rank, addr, dims, strides, box, elem, il, sw, l2, oob);
}
cudaError_t cudaGetDriverEntryPoint(const char *sym, void **fn, unsigned long long flags,
                                    enum cudaDriverEntryPointQueryResult *q) {
  const bool id = strcmp(sym, "cuStreamGetId") == 0;
  if (id ? no_ids : strcmp(sym, "cuTensorMapEncodeTiled") != 0) return fake_lane_entry_point(sym, fn, flags, q);
  *fn = id ? reinterpret_cast<void *>(&fake_stream_id) : reinterpret_cast<void *>(&locked_encode);
  if (q) *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}

// The shared decode's launches are recorded; while `meet` is set each waits until that
// many are under way at once, or half a second.
static std::mutex shared_mu;
static std::condition_variable shared_cv;
static std::vector<std::pair<pad::SharedParams, cudaStream_t>> shared_launches;
static int now_inside = 0, most_inside = 0, meet = 0;
namespace pad {
cudaError_t launch_shared(const SharedParams &p, int, bool, cudaStream_t s) {
  std::unique_lock<std::mutex> lock(shared_mu);
  shared_launches.push_back({p, s});
  most_inside = std::max(most_inside, ++now_inside);
  shared_cv.notify_all();
  if (meet > 0) shared_cv.wait_for(lock, std::chrono::milliseconds(500), [] { return most_inside >= meet; });
  --now_inside;
  return cudaSuccess;
}
}  // namespace pad

struct SharedProblem : Problem {
  pad_tensor table;
  explicit SharedProblem(int64_t B_ = 4) : Problem(B_, 8, 2, 128, 16, 8) {
    table = tensor(fake::device_buffer(4 * 4), PAD_I32, {4});
  }
  pad_status shared(void *stream, void *ws = nullptr, size_t bytes = 0) {
    return pad_decode_shared(&q, &k, &v, &table, &tables, &lens, 0.125f, nullptr, &out, &lse, ws, bytes, stream);
  }
};

static void each_thread_its_default_stream() {
  Problem p(2, 8, 2, 128, 16, 32);
  SharedProblem s;
  void *per_thread = cudaStreamPerThread;
  // all threads alive at once, so that their ids differ
  std::mutex mu;
  std::condition_variable cv;
  int turn = 0;
  std::vector<std::thread> threads;
  for (int i = 0; i < 3; ++i)
    threads.emplace_back([&, i] {
      std::unique_lock<std::mutex> lock(mu);
      cv.wait(lock, [&] { return turn == i; });
      for (int again = 0; again < 2; ++again) {
        CHECK(p.decode(4, per_thread) == PAD_OK, "decode: %s", pad_last_error());
        CHECK(s.shared(per_thread) == PAD_OK, "shared: %s", pad_last_error());
      }
      ++turn;
      cv.notify_all();
      cv.wait(lock, [&] { return turn == 3; });
    });
  for (auto &t : threads) t.join();
  CHECK(fake::launches.size() == 6 && shared_launches.size() == 6, "launches");
  for (size_t i = 0; i < 6; ++i)
    for (size_t j = 0; j < i; ++j) {
      const bool same = i / 2 == j / 2;
      CHECK((fake::launches[i].p.o_part == fake::launches[j].p.o_part) == same, "partials of threads %zu, %zu", i / 2, j / 2);
      CHECK((fake::launches[i].p.counters == fake::launches[j].p.counters) == same, "counters of %zu, %zu", i / 2, j / 2);
      CHECK((shared_launches[i].first.o_part == shared_launches[j].first.o_part) == same, "scratch of %zu, %zu", i / 2, j / 2);
    }
  CHECK(pad_release_workspace(-1) == PAD_OK && fake::library_live() == 0, "released");
}

static int device_syncs() {
  int n = 0;
  for (auto &e : fake::events) n += e == "devsync";
  return n;
}

static void a_handle_that_comes_back() {
  SharedProblem s;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(0x70);
  CHECK(s.shared(stream) == PAD_OK && s.shared(stream) == PAD_OK && device_syncs() == 0, "the same stream waits for nothing");
  stream_ids[stream] = 77;  // destroyed, and created again with work of the old one still queued
  CHECK(s.shared(stream) == PAD_OK && device_syncs() == 1, "scratch waited for");
  // a graph of this stream keeps its buffer when the handle goes to a third one
  fake::capturing = true;
  CHECK(s.shared(stream) == PAD_OK, "%s", pad_last_error());
  fake::capturing = false;
  stream_ids[stream] = 78;
  CHECK(s.shared(stream) == PAD_OK, "%s", pad_last_error());
  const size_t last = shared_launches.size() - 1;
  CHECK(shared_launches[last].first.o_part != shared_launches[last - 1].first.o_part, "the graph's buffer");
  CHECK(fake::find(shared_launches[last - 1].first.o_part) != nullptr, "the graph's buffer is still there");
  CHECK(pad_release_workspace(-1) == PAD_OK && fake::library_live() == 0, "released");
}

// Threads one after another: a new one may get an ended one's id, and its default
// stream is another all the same.
static void a_thread_id_that_comes_back() {
  Problem p(2, 8, 2, 128, 16, 32);
  SharedProblem s;
  std::thread::id id;
  int reused = 0;
  for (int i = 0; i < 8; ++i) {
    std::thread([&] {
      const bool same = std::this_thread::get_id() == id;
      id = std::this_thread::get_id();
      const int before = device_syncs();
      CHECK(p.decode(4, cudaStreamPerThread) == PAD_OK, "%s", pad_last_error());
      CHECK(!same || device_syncs() == before + 2, "partials and counters of an ended thread are waited for");
      CHECK(s.shared(cudaStreamPerThread) == PAD_OK, "%s", pad_last_error());
      CHECK(!same || device_syncs() == before + 3, "scratch of an ended thread is waited for");
      const int after = device_syncs();
      CHECK(p.decode(4, cudaStreamPerThread) == PAD_OK && s.shared(cudaStreamPerThread) == PAD_OK && device_syncs() == after,
            "its own is not");
      reused += same;
    }).join();
  }
  CHECK(reused > 0, "no thread id came back here");
  CHECK(pad_release_workspace(-1) == PAD_OK && fake::library_live() == 0, "released");
}

// Asking for the id of a stream under capture would end the capture.
static void under_capture_no_id_is_asked_for() {
  Problem p(2, 8, 2, 128, 16, 32);
  SharedProblem s;
  for (cudaStream_t stream : {reinterpret_cast<cudaStream_t>(0x70), cudaStreamPerThread}) {
    CHECK(p.decode(4, stream) == PAD_OK && s.shared(stream) == PAD_OK, "%s", pad_last_error());
    fake::capturing = true;
    const int before = ids_asked;
    CHECK(p.decode(4, stream) == PAD_OK && s.shared(stream) == PAD_OK && ids_asked == before, "asked");
    fake::capturing = false;
  }
  CHECK(pad_release_workspace(-1) == PAD_OK && fake::library_live() == 0, "released");
}

// How many calls of two threads are between their two kernels at once.
template <class Call>
static int at_once(Call call) {
  most_inside = 0;
  meet = 2;
  std::thread a([&] { CHECK(call(0) == PAD_OK, "%s", pad_last_error()); });
  std::thread b([&] { CHECK(call(1) == PAD_OK, "%s", pad_last_error()); });
  a.join();
  b.join();
  meet = 0;
  return most_inside;
}

static void only_one_streams_calls_wait_for_one_another() {
  SharedProblem p[2];
  void *streams[2] = {reinterpret_cast<void *>(0x70), reinterpret_cast<void *>(0x80)};
  pad_shared_plan plan;
  CHECK(pad_decode_shared_plan(4, 8, 2, 128, 16, 8, 4, PAD_BF16, 0, &plan) == PAD_OK, "plan");
  const size_t bytes = (size_t)plan.workspace_bytes;
  void *ws[2] = {fake::device_buffer(bytes), fake::device_buffer(bytes)};
  for (int i = 0; i < 2; ++i) CHECK(p[i].shared(streams[i]) == PAD_OK, "%s", pad_last_error());  // scratch exists
  CHECK(at_once([&](int i) { return p[i].shared(streams[i]); }) == 2, "two streams");
  CHECK(at_once([&](int i) { return p[i].shared(streams[0], ws[i], bytes); }) == 2, "workspaces of the callers");
  CHECK(at_once([&](int i) { return p[i].shared(streams[0]); }) == 1, "one stream's scratch");
  // a release waits for the call that holds the scratch
  meet = 2;
  most_inside = 0;
  std::thread call([&] { CHECK(p[0].shared(streams[0]) == PAD_OK, "%s", pad_last_error()); });
  {
    std::unique_lock<std::mutex> lock(shared_mu);
    shared_cv.wait(lock, [] { return now_inside == 1; });
  }
  std::thread release([&] { CHECK(pad_release_workspace(-1) == PAD_OK, "%s", pad_last_error()); });
  std::this_thread::sleep_for(std::chrono::milliseconds(100));
  {
    std::lock_guard<std::mutex> lock(shared_mu);
    CHECK(now_inside == 1, "the call is over already");
    CHECK(fake::find(shared_launches.back().first.o_part) != nullptr, "freed under a call");
  }
  call.join();
  release.join();
  meet = 0;
  CHECK(fake::library_live() == 0, "released");
  CHECK(p[0].shared(streams[0]) == PAD_OK && pad_release_workspace(-1) == PAD_OK && fake::library_live() == 0, "again");
}

int main(int argc, char **argv) {
  const std::string what = argc > 1 ? argv[1] : "";
  no_ids = argc > 2 && std::string(argv[2]) == "no-ids";
  if (what == "threads") each_thread_its_default_stream();
  else if (what == "reuse") a_handle_that_comes_back();
  else if (what == "thread-reuse") a_thread_id_that_comes_back();
  else if (what == "capture") under_capture_no_id_is_asked_for();
  else if (what == "locks") only_one_streams_calls_wait_for_one_another();
  else return 2;
  if (failures) return 1;
  puts("clean");
  for (const auto &a : std::vector<fake::Alloc>(fake::allocs)) free(a.base);
  return 0;
}
