// Beam search on the device: launch arguments of the candidates' selection and of the states' reordering.
#pragma once
#include "oscar_internal.h"

namespace oscar {

constexpr int kMaxBeams = 64;       // beams of an item
constexpr int kMaxCandidates = 64;  // candidates taken of an item
constexpr int kMaxVocab = 1 << 24;
constexpr int kBeamUnit = 1024;     // logits that a warp looks through at a time

// Units of a row; the workspace holds (maximum, sum of exponentials) of each.
OSCAR_HD inline int beam_units(int vocab) { return (vocab + kBeamUnit - 1) / kBeamUnit; }
inline size_t beam_ws_bytes(int batch, int beams, int vocab) { return (size_t)batch * beams * beam_units(vocab) * 2 * sizeof(float); }

struct BeamArgs {
  const void* logits;
  long long stride;              // elements between rows
  int dtype;
  const float* scores;           // [batch][beams]
  const uint8_t* finished;       // [batch][beams], or null
  int pad_token;
  int batch, beams, vocab, n_out;
  float* out_scores;             // [batch][n_out]
  int* out_tokens;
  int* out_parents;
  int* status;
  float* part;                   // [batch * beams][units][2]
};

struct ReorderArgs {
  Geom g;
  const int* parents;            // [batch][beams]
  int batch, beams;
  const int* block_table;
  int bt_stride;
  const int* seq_lens;
  const int* req_slot;
  int* new_block_table;
  int* new_seq_lens;
  int* new_req_slot;
  uint16_t* tail;                // [layers][max_req][Hkv][2][P][D]
  int* status;
};

int launch_beam_units(const BeamArgs& a, void* stream, bool pdl);
int launch_beam_pick(const BeamArgs& a, void* stream, bool pdl);
int launch_kv8_reorder(const ReorderArgs& a, void* stream, bool pdl);

}  // namespace oscar
