// host_check_streams.cpp -- in which order the library clears the workspaces that it allocates
// (barrier words, tile counters, ready counters, status) and launches the kernels that poll them,
// without a GPU: the program takes the place of the few runtime calls that the all-reduce makes
// and keeps account of what each stream has been given.
//
// The rule: when a kernel is launched on a stream, everything that the library has allocated in calls
// on that stream has been cleared on it, or elsewhere and waited for by the host.  hipMemset clears in the order of the
// null stream, does not wait on the host for device memory, and a stream made with
// hipStreamNonBlocking is not ordered behind the null stream.
#include <hip/hip_runtime_api.h>

#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <vector>

#include "ra.h"

namespace ra {
hipError_t launch_fill_u32(uint32_t* dst, uint32_t value, int64_t count, hipStream_t s);
}

namespace {

int failures = 0, launches = 0, fills = 0;
const char* doing = "";

struct Memory {
  size_t bytes;
  bool cleared, settled;      // settled: the host has waited for the clear
  hipStream_t on;             // the stream that cleared it
  hipStream_t of;             // the stream whose call allocated it
};
std::map<char*, Memory> live;
const void* fill_kernel = nullptr;
hipStream_t calling = nullptr;     // the stream of the call that is being made
struct Config {
  dim3 grid, block;
  size_t lds;
  hipStream_t s;
};
std::vector<Config> configs;

void wrong(const char* what) {
  std::printf("FAIL %s: %s\n", doing, what);
  ++failures;
}

// The allocation that holds all of [p, p + bytes), or null.
Memory* holder(void* p, size_t bytes) {
  char* at = static_cast<char*>(p);
  auto it = live.upper_bound(at);
  if (it == live.begin()) return nullptr;
  --it;
  return at + bytes <= it->first + it->second.bytes ? &it->second : nullptr;
}

void settle(hipStream_t s) {
  for (auto& m : live)
    if (m.second.on == s) m.second.settled = true;
}

void clear(void* p, int value, size_t bytes, hipStream_t s) {
  Memory* m = holder(p, bytes);
  if (!m) return wrong("a clear outside the allocations");
  std::memset(p, value, bytes);
  if (bytes < m->bytes) return;
  m->cleared = value == 0;
  m->settled = false;
  m->on = s;
}

}  // namespace

// ---------------------------------------------------------------- the runtime's calls

extern "C" {
hipError_t hipGetDevice(int* dev) { return *dev = 0, hipSuccess; }
hipError_t hipGetLastError() { return hipSuccess; }
hipError_t hipStreamIsCapturing(hipStream_t, hipStreamCaptureStatus* s) { return *s = hipStreamCaptureStatusNone, hipSuccess; }
hipError_t hipDeviceGetAttribute(int* v, hipDeviceAttribute_t a, int) {
  return *v = a == hipDeviceAttributeMultiprocessorCount ? 256 : 100000, hipSuccess;
}
hipError_t hipOccupancyMaxActiveBlocksPerMultiprocessor(int* n, const void*, int threads, size_t) {
  return *n = 2048 / threads, hipSuccess;
}
hipError_t hipMalloc(void** p, size_t bytes) {
  *p = std::malloc(bytes);
  std::memset(*p, 0xAB, bytes);             // what earlier owners left
  live[static_cast<char*>(*p)] = {bytes, false, false, nullptr, calling};
  return hipSuccess;
}
hipError_t hipFree(void* p) {
  if (live.erase(static_cast<char*>(p)) != 1) wrong("freed what is no allocation");
  std::free(p);
  return hipSuccess;
}
hipError_t hipMemset(void* p, int value, size_t bytes) { return clear(p, value, bytes, nullptr), hipSuccess; }
hipError_t hipMemsetAsync(void* p, int value, size_t bytes, hipStream_t s) { return clear(p, value, bytes, s), hipSuccess; }
// Copies that the host waits for, in the order of the null stream.
hipError_t hipMemcpy(void* to, const void* from, size_t bytes, hipMemcpyKind) {
  settle(nullptr);
  std::memcpy(to, from, bytes);
  return hipSuccess;
}
hipError_t hipStreamSynchronize(hipStream_t s) { return settle(s), hipSuccess; }
hipError_t hipDeviceSynchronize() {
  for (auto& m : live) m.second.settled = true;
  return hipSuccess;
}
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t lds, hipStream_t s) {
  return configs.push_back({grid, block, lds, s}), hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* lds, hipStream_t* s) {
  const Config c = configs.back();
  configs.pop_back();
  *grid = c.grid, *block = c.block, *lds = c.lds, *s = c.s;
  return hipSuccess;
}
hipError_t hipLaunchKernel(const void* f, dim3, dim3, void** args, size_t, hipStream_t s) {
  if (!fill_kernel) return fill_kernel = f, hipSuccess;        // main() begins with one
  if (f == fill_kernel) {
    ++fills;
    uint32_t* dst = *static_cast<uint32_t**>(args[0]);
    const uint32_t value = *static_cast<uint32_t*>(args[1]);
    const int64_t count = *static_cast<int64_t*>(args[2]);
    clear(dst, (int)value, (size_t)count * 4, s);
    return hipSuccess;
  }
  if (s == nullptr) return hipSuccess;      // the probe of the workgroups' places
  ++launches;
  if (s != calling) wrong("a kernel is launched on another stream");
  for (auto& m : live) {
    if (m.second.of != s) continue;
    if (!m.second.cleared) wrong("a kernel is launched before a workspace is cleared");
    else if (!m.second.settled && m.second.on != s) wrong("a kernel is launched that is not ordered behind a workspace's clear");
  }
  return hipSuccess;
}
}  // extern "C"

namespace {

void expect(int got, int want) {
  if (got == want) return;
  std::printf("FAIL %s: %d, expected %d (%s)\n", doing, got, want, ra_last_error());
  ++failures;
}

hipStream_t stream(int i) { return reinterpret_cast<hipStream_t>(uintptr_t(0x1000) + 64 * i); }

void* bufs[8];

int reduce(int algo, const ra_options& o, hipStream_t s) {
  calling = s;
  return ra_allreduce_ex(bufs, 8, 50000, RA_FLOAT32, RA_SUM, algo, &o, s);
}

}  // namespace

int main() {
  for (int r = 0; r < 8; ++r) bufs[r] = reinterpret_cast<void*>(uintptr_t(0x7f0000000000ull) + uintptr_t(r) * (1 << 20));
  // which kernel fills
  uint32_t word;
  expect(ra::launch_fill_u32(&word, 0u, 1, nullptr), hipSuccess);

  ra_options o;
  std::memset(&o, 0, sizeof o);
  doing = "flag-driven ring, the first call of the process";
  expect(reduce(RA_ALGO_RING_PIPELINED_FLAGS, o, stream(1)), RA_OK);
  doing = "flag-driven ring, the first call on its stream";
  expect(reduce(RA_ALGO_RING_PIPELINED_FLAGS, o, stream(2)), RA_OK);
  doing = "channels, the first call on its stream";
  ra_options channels = o;
  channels.channels = 8;
  expect(reduce(RA_ALGO_RING_CHANNELS, channels, stream(3)), RA_OK);
  doing = "flag-driven ring behind channels";
  expect(reduce(RA_ALGO_RING_PIPELINED_FLAGS, o, stream(3)), RA_OK);
  doing = "a grid, the first call on its stream";
  ra_options grid = o;
  grid.grid = 40;
  for (int algo : {RA_ALGO_RING_STEP, RA_ALGO_RING_BIDIR, RA_ALGO_TREE, RA_ALGO_HIER})
    expect(reduce(algo, grid, stream(4 + algo)), RA_OK);
  doing = "resident copy, the first call on its stream";
  calling = stream(20);
  expect(ra_stream_copy_resident(bufs[0], bufs[1], 1 << 16, 64, stream(20)), RA_OK);
  doing = "more ready counters than the stream has";
  ra_options small = o;
  small.slice_elems = 256;
  small.grid = 64;
  calling = stream(2);
  expect(ra_allreduce_ex(bufs, 8, 250000, RA_FLOAT32, RA_SUM, RA_ALGO_RING_PIPELINED_FLAGS, &small, stream(2)), RA_OK);
  small.slice_elems = 32;
  expect(ra_allreduce_ex(bufs, 8, 250000, RA_FLOAT32, RA_SUM, RA_ALGO_RING_PIPELINED_FLAGS, &small, stream(2)), RA_OK);
  doing = "renewed ready counters";
  ra_options renew = o;
  renew.flags = RA_FLAG_RENEW_COUNTERS;
  for (int k = 0; k < 3; ++k) expect(reduce(RA_ALGO_RING_PIPELINED_FLAGS, renew, stream(1)), RA_OK);
  doing = "reduce-scatter and all-gather, the first calls on their stream";
  calling = stream(21);
  expect(ra_reduce_scatter_ex(bufs, 8, 50000, RA_FLOAT32, RA_SUM, RA_ALGO_RING_PIPELINED_FLAGS, &o, stream(21)), RA_OK);
  expect(ra_all_gather_ex(bufs, 8, 50000, RA_FLOAT32, RA_ALGO_RING_PIPELINED_FLAGS, &o, stream(21)), RA_OK);

  // a wait that ran out: its status is reported once, its header cleared, and the next call goes
  doing = "the call behind a status that was reported";
  std::map<char*, Memory> before = live;
  expect(reduce(RA_ALGO_RING_CHANNELS, channels, stream(22)), RA_OK);
  char* header = nullptr;
  for (auto& m : live)
    if (!before.count(m.first)) header = m.first;
  if (!header) {
    wrong("no workspace was allocated");
  } else {
    *reinterpret_cast<uint32_t*>(header) = RA_ERR_TIMEOUT;     // the status comes first
    live[header].cleared = false;
    expect(ra_stream_status(stream(22)), RA_ERR_TIMEOUT);
    expect(ra_stream_status(stream(22)), RA_OK);
    expect(reduce(RA_ALGO_RING_CHANNELS, channels, stream(22)), RA_OK);
  }
  if (launches < 16) wrong("fewer launches than calls");
  std::printf(failures ? "FAILED %d\n" : "PASSED (%d launches, %d fills)\n", failures ? failures : launches, fills);
  return failures != 0;
}
