// 8-bit paged cache: geometry, launch arguments and launchers (host and device).
#pragma once
#include "oscar_internal.h"

namespace oscar {

constexpr int kKv8Int8 = 0;
constexpr int kKv8E4m3 = 1;
// A block whose largest finite magnitude is below this is stored as zeros with scale 0
// (2^-100: scale and quotients of larger ones stay normal float32 numbers).
constexpr float kKv8Smallest = 7.888609052210118e-31f;
// Attention walks whole pages in stages of 64 tokens, or of 128 where that is no more than 16 KB of codes and a quarter of it
// lies in one page.
OSCAR_HD constexpr int kv8_stage_tokens(int D, int P) { return D == 64 && P >= 32 ? 128 : 64; }

// Byte layout of one (layer, page, kv head) block:
//   K codes [P][D] | V codes [P][D] | K scale, V scale (float32), 8 unused bytes | K lo [D] | K hi [D] | pad to 128
// Token rows are D bytes in channel order, but the 16-byte chunks of each 128-byte line
// of a code section are stored at (chunk ^ turn): turn = 4 (t & 1) for K at D = 128 (0 at
// D = 64) and 2 ((t >> 1) & 3) for V, t the chunk's token.  With it the decode kernel's
// fragment loads from shared memory touch every bank once.
struct Kv8Geom {
  int P, D, Hkv;
  OSCAR_HD size_t v_off() const { return (size_t)P * D; }
  OSCAR_HD size_t scale_off() const { return 2 * (size_t)P * D; }
  OSCAR_HD size_t lo_off() const { return scale_off() + 16; }
  OSCAR_HD size_t hi_off() const { return lo_off() + D; }
  OSCAR_HD size_t block_bytes() const { return (hi_off() + D + 127) & ~size_t(127); }
  OSCAR_HD size_t page_bytes() const { return (size_t)Hkv * block_bytes(); }
};

OSCAR_HD inline Kv8Geom kv8_geom(const Geom& g) { return Kv8Geom{g.P, g.D, g.Hkv}; }
inline size_t kv8_pool_bytes(const Geom& g) { return (size_t)g.L * g.num_pages * kv8_geom(g).page_bytes(); }
// bf16 elements of one (layer, request slot) tail region: [Hkv][2][P][D]
OSCAR_HD inline size_t kv8_tail_req_elems(const Geom& g) { return (size_t)g.Hkv * 2 * g.P * g.D; }
inline size_t kv8_tail_bytes(const Geom& g) { return (size_t)g.L * g.max_req * kv8_tail_req_elems(g) * 2; }

struct Kv8WriteArgs {
  Geom g;
  int fmt, layer;
  const void* K;
  const void* V;
  long long k_stride, v_stride;  // elements between tokens
  int dtype;
  const int* cu_seqlens;         // null: append (one token per request)
  const int* start_pos;          // cached tokens of each request before the call
  int batch, total_tokens;
  const int* block_table;
  int bt_stride;
  const int* req_slot;
  uint8_t* pool;
  uint16_t* tail;
  int* status;
};

struct Kv8DecodeWs {
  int stages_per_split;  // stages of one split CTA
  int max_splits;        // splits of a request, one at least
  size_t total;          // bytes: partials [batch][Hq][max_splits][D + 4] float32
};

// Tokens by which the shared pages of a group are split.
constexpr int kPrefixUnit = 128;

// Requests that share their first pages, group by group (n = 0: none do).
struct Kv8Groups {
  const int* starts;             // [n + 1]: group i holds requests starts[i] .. starts[i + 1] - 1
  const int* shared;             // [n]: pages that a group's requests share
  int n, max_shared;             // max_shared bounds shared
  int max_own;                   // bounds the tokens behind them
  int units_per_split;           // units of tokens of one CTA of the prefix kernel
  int max_tiles;                 // row tiles of all groups, at most
  int slots;                     // partials of a row for the prefix: places 0 .. slots - 1
};

struct Kv8DecodeArgs {
  Geom g;
  int fmt, layer;
  const void* q;
  long long q_stride;            // elements between requests
  int q_dtype;
  void* out;
  int out_dtype;
  const int* page_idx;           // sparse: [batch][Hkv][n_select] logical pages, ascending, -1 after the last; dense: null
  int n_select;
  const int* block_table;
  int bt_stride;
  const int* seq_lens;
  const int* req_slot;
  int batch, max_seq;
  const uint8_t* pool;
  const uint16_t* tail;
  int* status;
  float* part;
  Kv8DecodeWs wl;
  Kv8Groups groups;              // the pages before shared[] are another kernel's
  int splits;                    // CTAs of a request and kv head; wl.max_splits of them, or less where the prefix has places
};

struct Kv8SelectArgs {
  Geom g;
  int fmt, layer;
  const void* q;
  long long q_stride;
  int q_dtype;
  const int* block_table;
  int bt_stride;
  const int* seq_lens;
  int batch, max_seq;
  int keep_first, keep_last, n_select;
  int* page_idx;
  const uint8_t* pool;
  int* status;
  uint8_t* ws;
  int max_pages;                 // max_seq / P
};

// Host-side lists that a kernel takes by value: they need no device buffer and no copy.  A call with
// more entries launches once per list of kMostPairs; a short list goes in a short argument, which
// takes the host less time to hand over.
constexpr int kMostPairs = 1000, kFewPairs = 60;
template <int N>
struct IntPairs {
  int n;
  int src[N];  // ascending
  int dst[N];
};

Kv8DecodeWs kv8_plan(const Geom& g, int batch, long long max_pages);
// the same for requests in groups: the plan of their own parts, with room for the prefixes' partials
Kv8DecodeWs kv8_shared_plan(const Geom& g, int batch, int n_groups, int max_shared, int max_own, Kv8Groups* groups, int* own_splits);
// bytes that serve every call of at most so many requests and groups with these bounds
size_t kv8_shared_ws_bytes(const Geom& g, int batch, int n_groups, int max_shared, int max_own);
size_t kv8_select_ws_bytes(const Geom& g, int batch, int max_seq);

int launch_kv8_write(const Kv8WriteArgs& a, void* stream, bool pdl);
int launch_kv8_decode(const Kv8DecodeArgs& a, void* stream, bool pdl);
int launch_kv8_shared_prefix(const Kv8DecodeArgs& a, void* stream, bool pdl);
int launch_kv8_combine(const Kv8DecodeArgs& a, void* stream, bool pdl);
int launch_kv8_select(const Kv8SelectArgs& a, void* stream, bool pdl);
// rows [0, n_rows) of the src slot's tail to every dst slot (n <= kMostPairs of them), in every layer
int launch_kv8_fork_tail(const Geom& g, uint16_t* tail, int src, const int* dst, int n, int n_rows, void* stream);
// pool: [layers][num_pages][page_bytes]; page src[i] to page dst[i] in every layer (n <= kMostPairs)
int launch_copy_pages(uint8_t* pool, int layers, int num_pages, size_t page_bytes, const int* src, const int* dst, int n,
                      void* stream);
// block-table entries equal to src[i] (ascending) become dst[i] (n <= kMostPairs)
int launch_remap_table(int* table, int rows, int cols, const int* src, const int* dst, int n, void* stream);

}  // namespace oscar
