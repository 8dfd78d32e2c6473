// mac_beam.cuh -- parameter blocks and launchers of the calls of beam search:
// the selection over beams and vocabulary, and the slots' new histories.
#pragma once

#include "mac_batch.cuh"

namespace mac {

constexpr int kMaxBeams = MAC_MAX_BEAMS;
constexpr int kMaxPicks = MAC_MAX_CANDIDATES;  // candidates that a selection returns per group
constexpr int kMaxVocab = 1 << 20;
// The selection's scan cuts a row into at most kMaxPieces pieces, of a number of
// steps: 16 bytes for each thread of a CTA.
constexpr int kScanThreads = 256, kMaxPieces = 64;

struct SelectParams {
  int S, n, V, n_out, placed, end;
  int steps, segs;                // of a piece; pieces of a row
  unsigned long long beam_inv;     // 2^40 / (n_out segs), rounded up: i times it, shifted, is the quotient
  int64_t stride;                 // elements between rows
  const void *logits;
  const float *scores;            // [S]
  const int32_t *done;            // [S] or null
  float *scores_out;              // [S / n][n_out]
  int32_t *parent, *token, *done_out;
  float2 *ml;                     // [S][segs] maximum and sum of exp of a CTA's logits
  unsigned long long *keys;       // [S][n_out][segs] its best ones; 0: none
  uint32_t *counts;               // [S / n] CTAs of a group that are done; zero before and after a call
  uint32_t *status;
};

// A slot's move: what a layer copies into it.
struct Move {
  int src;                        // slot copied from, -1: nothing to copy
  int first, last;                // positions whose ring entries may differ
  int len;                        // tokens of the new history
  int page_from, page_to, rows;   // a parted page: its first `rows` rows are copied
  int unused;
};
static_assert(sizeof(Move) == 32, "two 16-byte words");

struct ReorderParams {
  int S, n, paged;
  int64_t limit;                  // longest length of a slot
  int max_pages, n_pages;
  int32_t *table, *free_pages;
  const int32_t *n_free_in;
  int32_t *n_free_out;
  const int32_t *parent, *len_in, *shared_in;
  int32_t *len_out, *shared_out;
  Move *moves;
  uint32_t *status;
};

struct StateParams {
  int S, n, Hq, Hkv, K, es, paged;
  int64_t capacity;               // contiguous: tokens per slot
  int n_pages;
  const Move *moves;
  int32_t *pos;                   // the rings, or null
  uint8_t *q;
  float *o, *lse;
  uint8_t *k, *v;                 // the cache, or null
  uint32_t *status;
};

cudaError_t launch_reorder(const ReorderParams &p, cudaStream_t s);
cudaError_t launch_state(const StateParams &p, int sms, cudaStream_t s);
cudaError_t launch_select(const SelectParams &p, int dtype, cudaStream_t s);

}  // namespace mac
