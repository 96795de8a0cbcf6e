// Plan records of the prompt attention, shared by its planner (prompt_plan.cpp)
// and its kernels (prompt_attn.cu).
#pragma once

#include "gk_internal.h"

namespace gk {

struct PromptReqDev {
  int64_t hot_row;     // first row of the slab in the HOT pool seen as rows of d elements
  int32_t lp;          // HOT tokens
  int32_t ctx;         // COLD tokens
  int32_t n;           // new tokens
  int32_t t0;          // its first row of the packed tensors
  int32_t nt_hot;      // 128-key tiles of the HOT tokens ...
  int32_t nt_cold;     // ... and of the COLD tokens
  int32_t row;         // row of the block table
  int32_t pad0;
};

struct PromptItemDev {
  int32_t req;
  int32_t head;        // KV head
  int32_t tok0;        // first of its 2 * floor(128 / g) tokens
  int32_t tile0;       // key tiles [tile0, tile0 + ntile) of the request: HOT, COLD, new
  int32_t ntile;
  int32_t entry;       // partial state, -1 = the item covers every key and writes the output
  int32_t part_row;    // its first row: a state has one for each row of the item's tokens, token by token
  int32_t pad0;
};

struct PromptJoinDev { // 32 rows of a block whose keys several items cover
  int32_t req;
  int32_t head;
  int32_t tok0;        // first token of the block
  int32_t row0;        // first of the 32 rows, counted from the block's first
  int32_t own0, own_n; // first row of the partial states of the block's own items, and how many states
  int32_t hot0, hot_n; // the same of the stacked prefix items of this head (hot_n states per block), 0 = none
  int32_t hot_tok;     // the block's first token, counted from the first token of the stacked requests
  int32_t hot_len;     // tokens of the stacked requests
};

struct PromptPlan {
  Pool* pool = nullptr;
  gk_prompt_plan_summary summary{};
  int32_t n_requests = 0;                // reqs past them are stacked runs of requests
  int64_t tokens = 0;
  bool any_hot = false, any_cold = false;
  int32_t max_blocks = 0;                // blocks that the longest COLD context needs
  std::vector<PromptReqDev> reqs;
  std::vector<PromptItemDev> items;      // grouped by CTA
  std::vector<int32_t> cta_begin;        // [CTAs + 1]
  std::vector<PromptJoinDev> joins;
  int32_t n_entries = 0;
  int64_t part_rows = 0;                 // rows of all partial states
  uint8_t hot_maps[256] = {};            // tensor maps of the HOT pool's K and V (any_hot)
  void* d_buf = nullptr;
  void* h_stage = nullptr;
  cudaEvent_t upload_done = nullptr;
  bool staged = false;
  size_t d_bytes = 0;
  size_t off_reqs = 0, off_items = 0, off_begin = 0, off_joins = 0;
  float* d_part_o = nullptr;             // [rows][d]
  float* d_part_l = nullptr;             // [rows] (log2)
  size_t part_cap = 0;                   // rows that both hold
  bool uploaded = false;
};

// the tensor maps of a pool's HOT K and V, 128 bytes each
int encode_hot_maps(const gk_pool_config* cfg, uint8_t* out);
int launch_prompt(const LaunchCommon& lc, void* stream, int32_t layer, const gk_prompt_batch* b, const PromptPlan* pl);

}  // namespace gk

struct gk_prompt_plan {
  gk::PromptPlan impl;
};
