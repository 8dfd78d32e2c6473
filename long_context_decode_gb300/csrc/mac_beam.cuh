// mac_beam.cuh -- parameter blocks and launchers of the calls of beam search:
// the selection over beams and vocabulary, and the slots' new histories.
#pragma once

#include "mac_batch.cuh"

namespace mac {

constexpr int kMaxBeams = MAC_MAX_BEAMS;
constexpr int kMaxPicks = MAC_MAX_CANDIDATES;  // candidates that a selection returns per group
constexpr int kMaxVocab = 1 << 20;
// A CTA of the selection's scan takes kScanThreads * per logits of a row, per one of 8, 16, 32.
constexpr int kScanThreads = 256, kScanLeast = 8;

struct SelectParams {
  int S, n, V, n_out, placed, end;
  int per, segs;                  // logits per thread, CTAs per row
  int64_t stride;                 // elements between rows
  const void *logits;
  const float *scores;            // [S]
  const int32_t *done;            // [S] or null
  float *scores_out;              // [S / n][n_out]
  int32_t *parent, *token, *done_out;
  float2 *ml;                     // [S][segs] maximum and sum of exp of a CTA's logits
  unsigned long long *keys;       // [S][segs][n_out] its best ones; 0: none
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
