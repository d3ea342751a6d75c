// The handle behind include/tok.h and the helpers that every entry point
// shares: error messages, the current-device guard, allocations (which honour
// the failure hook of tok_debug_fail_alloc).
#pragma once
#include <algorithm>
#include <atomic>
#include <cstddef>
#include <cstdint>
#include <string>
#include <vector>

#include "../../include/tok.h"
#include "tok_common.cuh"

namespace tokgb {

// The vocabulary's bytes on the device: token t has bytes[off[t] .. off[t + 1]),
// and, for walking many tokens at once, the tokens sorted by their bytes in
// groups of up to 32 that begin alike.  Group g: its first `prefix` bytes (at
// most 8; none, but for a look at the first one, where they would end inside
// a code point) are in head; lane i's token is id[32 g + i] (NO_TOKEN: none) with
// rest[32 g + i] bytes more, four per word, words[at + 32 w + i].  kinds has a
// bit for each kind of byte (byte_kind) among these, group_kinds for the
// whole group.
struct TokenGroup {
  unsigned long long head;  // the first byte lowest
  uint32_t prefix;
  uint32_t at;
};

struct DevTokens {
  const uint8_t* bytes;
  const uint32_t* off;
  uint32_t n;
  uint32_t n_groups;
  const TokenGroup* group;
  const uint32_t* words;
  const uint32_t* id;
  const uint32_t* kinds;
  const uint32_t* group_kinds;
  const uint32_t* rest;   // bytes | kind of the first one << 16 | how many of that kind it begins with << 21
};
constexpr uint32_t MOST_RUN = 2047;  // of those

// Kinds of bytes, such that what a grammar treats apart is often of different
// kinds; well-formed UTF-8 sequences of several bytes are one of their own.
constexpr uint32_t KIND_SEQUENCE = 29;
inline uint32_t byte_kind(uint8_t b) {
  if (b >= 0x80) return 28;
  if (b == 0x7f) return 27;
  if (b >= '0' && b <= '9') return b == '0' ? 8 : 9;
  if (b >= 'a' && b <= 'z') return b <= 'f' ? 10 : 11;
  if (b >= 'A' && b <= 'Z') return b <= 'F' ? 12 : 13;
  switch (b) {
    case '\t': return 1;
    case '\n': return 2;
    case '\r': return 3;
    case ' ': return 4;
    case '"': return 5;
    case '\\': return 6;
    case '\'': return 7;
    case '_': return 14;
    case '-': return 15;
    case '.': return 16;
    case ',': return 17;
    case ':': return 18;
    case ';': return 19;
    case '/': return 20;
    case '(': case ')': return 21;
    case '[': case ']': return 22;
    case '{': case '}': return 23;
    case '<': case '=': case '>': return 24;
    case '@': case '#': case '$': case '`': case '?': return 26;
  }
  return b < 0x20 ? 0 : 25;
}

}  // namespace tokgb

constexpr int N_STAGES = 3;  // kernels of an encode

constexpr unsigned long long kDefaultWaitNs = 4000000000ull;  // 4 s

struct tok_handle {
  int dev = 0;
  int n_sms = 1;
  int pattern = 0;
  cudaStream_t stream = nullptr;
  tokgb::DevVocab v{};
  // device allocations of the vocabulary
  tokgb::MergeEntry* d_table = nullptr;
  int32_t* d_byte_id = nullptr;
  uint16_t* d_tok_len = nullptr;
  uint16_t* d_max_left = nullptr;
  uint16_t* d_max_right = nullptr;
  tokgb::WholeEntry* d_whole = nullptr;
  unsigned long long* d_whole_tail = nullptr;
  uint64_t whole_tail_bytes = 0;
  uint32_t* d_pair_bits = nullptr;
  uint32_t n_whole = 0;
  uint64_t hash = 0;
  // host copy of the tokens' bytes (token t: vocab_bytes[vocab_off[t] .. vocab_off[t + 1]))
  std::vector<uint8_t> vocab_bytes;
  std::vector<uint64_t> vocab_off;
  // finished CTAs of a paged-cache call that completes in place; 0 between calls
  uint32_t* d_done = nullptr;
  // the tokens' bytes in the order the grammar kernels read them (laid out by
  // the first tok_grammar_load)
  tokgb::DevTokens tokens{};
  void* d_tokens = nullptr;
  // workspace
  tokgb::Workspace ws{};
  int32_t* d_out = nullptr;           // ids of host-side calls
  long long* d_off = nullptr;         // token byte offsets of host-side calls (allocated on first use)
  long long* d_items = nullptr;       // item starts of host-side batch calls
  long long* d_item_off = nullptr;
  uint64_t cap_items = 0;
  tokgb::DevStatus* h_status = nullptr;      // pinned
  long long* h_ustatus = nullptr;     // pinned, written by the device: code, ids, UTF-8 error offset
  long long* d_ustatus = nullptr;     // its device address
  long long* h_items = nullptr;       // pinned
  uint64_t cap_h_items = 0;
  uint32_t epoch = 0;
  std::string err;
  int64_t err_off = -1;
  uint32_t last_epoch = 0;            // epoch of the latest call
  uint64_t launches = 0;
  bool timing = false;
  cudaEvent_t ev[N_STAGES + 1] = {};
  float stage_ms[N_STAGES] = {};
  bool have_times = false;
  // test hook (tok_debug_fail_alloc): the allocation that fails, counted
  // from 1 = the next one; 0 = none
  uint32_t fail_alloc_in = 0;
  // limit of a device-side wait (the grid barriers of the BPE kernel), and
  // the test hook tok_debug_grid_wait: arrivals a grid barrier waits for
  // beyond the CTAs that come
  unsigned long long wait_ns = kDefaultWaitNs;
  uint32_t grid_extra = 0;
};

namespace tokgb {

struct DeviceGuard {
  int prev = -1;
  explicit DeviceGuard(int dev) {
    if (cudaGetDevice(&prev) == cudaSuccess && prev != dev) cudaSetDevice(dev);
    else prev = -1;
  }
  ~DeviceGuard() {
    if (prev >= 0) cudaSetDevice(prev);
  }
};

// Keep the message of a failure (of h, or of the last failed load when h is
// NULL) and return its code.
int fail(tok_handle* h, int code, const std::string& msg);
int cuda_fail(tok_handle* h, cudaError_t e, const char* what);

template <class T>
cudaError_t dalloc(T** p, size_t count) {
  return cudaMalloc(reinterpret_cast<void**>(p), std::max<size_t>(count, 1) * sizeof(T));
}

// true when the handle's failure hook says this allocation is the one that
// fails (it then stands in for a cudaMalloc that found the device full)
inline bool injected_failure(tok_handle* h) {
  return h->fail_alloc_in > 0 && --h->fail_alloc_in == 0;
}

// device allocation of a handle's buffers (workspace, items, offsets)
template <class T>
cudaError_t halloc(tok_handle* h, T** p, size_t count) {
  if (injected_failure(h)) {
    *p = nullptr;
    return cudaErrorMemoryAllocation;
  }
  return dalloc(p, count);
}

// pinned host allocation of a handle's buffers
template <class T>
cudaError_t halloc_pinned(tok_handle* h, T** p, size_t count) {
  if (injected_failure(h)) {
    *p = nullptr;
    return cudaErrorMemoryAllocation;
  }
  return cudaMallocHost(reinterpret_cast<void**>(p), std::max<size_t>(count, 1) * sizeof(T));
}

// Allow a kernel most of an SM's shared memory and clusters of 16 CTAs, once
// per device (the two calls cost about as much as a launch).
constexpr size_t MOST_SHARED = 200 * 1024;
template <auto Kernel>
cudaError_t allow_all(int dev) {
  static std::atomic<unsigned long long> done{0};
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)MOST_SHARED);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// Launch a kernel in clusters of `cluster` CTAs.
template <auto Kernel, class... Args>
cudaError_t launch_clusters(int dev, unsigned ctas, unsigned threads, unsigned cluster, size_t smem, cudaStream_t s,
                            const Args&... args) {
  const cudaError_t e = allow_all<Kernel>(dev);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  if (cluster > 1) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
  return cudaLaunchKernelEx(&cfg, Kernel, args...);
}

}  // namespace tokgb
