// Planner and entry points of the prompt attention: cuts a step's rows and keys
// into work items, balances them over the SMs and launches a layer.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>
#include <new>
#include <queue>

#include "prompt.h"

namespace gk {
namespace {

// What the planner weighs, in us on one SM of a GB300, read off runs of one item
// per SM: a 128-key tile of an item with two Q tiles and of one with one, an
// item's fixed cost, a join launch, and 32 joined rows.
constexpr double kTile2Us = 1.5;
constexpr double kTile1Us = 1.35;
constexpr double kItemUs = 3.5;
constexpr double kJoinLaunchUs = 4.0;
constexpr double kJoinUs = 1.0;
constexpr int32_t kMaxPieces = 16;      // items over one block's own keys, and over its stacked prefix
constexpr int32_t kBN = kPrefixTileN;

struct Run {              // neighbouring requests whose rows are stacked over one HOT prefix
  int32_t rec;            // its record in reqs
  int32_t n;              // tokens
  int32_t entry0 = 0;     // partial states: entry0 + (head * blocks + block) * pieces + piece
  int64_t row0 = 0;       // the first one's first row
  int32_t pieces = 1;
  int32_t blocks = 0;
};

struct Shape {            // one block of rows and its range of key tiles, before splitting
  int32_t req, tok0, tile0, ntile;
  bool two;
  int32_t run = -1, run_block = 0;   // a stacked prefix block
  bool joined = false;               // other items cover other keys of its rows
  int32_t hot_run = -1, hot_tok = 0; // its rows' stacked prefix
};

int32_t tiles(int64_t n) { return (int32_t)((n + kBN - 1) / kBN); }
double cost(const Shape& s, int32_t ntile) { return kItemUs + ntile * (s.two ? kTile2Us : kTile1Us); }
int32_t pieces_of(int32_t ntile, int32_t most) {
  return std::max(1, std::min(std::min(kMaxPieces, ntile), (ntile + most - 1) / most));
}

// longest-processing-time-first assignment of costs to `n` bins; the makespan, and each cost's bin
double balance(const std::vector<double>& cost, int n, std::vector<int32_t>* bin) {
  std::vector<int32_t> order(cost.size());
  for (size_t i = 0; i < order.size(); ++i) order[i] = (int32_t)i;
  std::stable_sort(order.begin(), order.end(), [&](int32_t a, int32_t b) { return cost[(size_t)a] > cost[(size_t)b]; });
  std::priority_queue<std::pair<double, int32_t>, std::vector<std::pair<double, int32_t>>, std::greater<>> q;
  for (int32_t b = 0; b < n; ++b) q.push({0.0, b});
  if (bin) bin->assign(cost.size(), 0);
  double top = 0;
  for (int32_t i : order) {
    auto [load, b] = q.top();
    q.pop();
    load += cost[(size_t)i];
    top = std::max(top, load);
    if (bin) (*bin)[(size_t)i] = b;
    q.push({load, b});
  }
  return top;
}

gk_status build_host(Pool* p, const gk_prompt_batch* b, PromptPlan* pl) {
  const gk_pool_config& c = p->cfg;
  const int32_t B = b->num_requests, G = p->g(), Hkv = c.num_kv_heads;
  const int32_t tpt = kPrefixTileM / G, bt = 2 * tpt;   // tokens per Q tile and per block
  if (B < 0) return fail(p, GK_ERR_INVALID, "num_requests < 0");
  if (B > 0 && !b->new_len) return fail(p, GK_ERR_INVALID, "batch host arrays missing");
  if ((b->prefix_hot_base == nullptr) != (b->prefix_len == nullptr))
    return fail(p, GK_ERR_INVALID, "prefix_hot_base and prefix_len go together");
  pl->pool = p;
  pl->n_requests = B;
  pl->reqs.clear();
  pl->items.clear();
  pl->cta_begin.assign(1, 0);
  pl->joins.clear();
  pl->n_entries = 0;
  pl->part_rows = 0;
  pl->any_hot = pl->any_cold = false;
  pl->max_blocks = 0;
  gk_prompt_plan_summary sum{};

  // ---- requests ------------------------------------------------------------------
  std::vector<int64_t> base_of((size_t)B, -1);
  int64_t T = 0, pairs = 0, kept = 0, table = 0;
  std::vector<std::pair<int64_t, int32_t>> used;
  for (int32_t r = 0; r < B; ++r) {
    PromptReqDev rq{};
    const int64_t base = b->prefix_hot_base ? b->prefix_hot_base[r] : -1;
    const int32_t lp = b->prefix_len ? b->prefix_len[r] : 0;
    rq.n = b->new_len[r];
    rq.ctx = b->context_len ? b->context_len[r] : 0;
    if (rq.n < 0 || rq.ctx < 0) return fail(p, GK_ERR_INVALID, "negative length");
    if ((int64_t)rq.ctx > (int64_t)b->max_blocks * c.cold_page_size)
      return fail(p, GK_ERR_INVALID, "context longer than the block-table row");
    if (base < 0) {
      if (lp != 0) return fail(p, GK_ERR_INVALID, "prefix_len must be 0 without a HOT prefix");
    } else {
      auto it = p->hot.live.find(base);
      if (it == p->hot.live.end() || it->second != lp)
        return fail(p, GK_ERR_INVALID, "request names a HOT prefix that is not live with that length");
      base_of[(size_t)r] = base;
      rq.lp = lp;
      rq.hot_row = base * c.num_layers * Hkv;
    }
    const int64_t keys = (int64_t)rq.lp + rq.ctx + rq.n;
    if (keys > INT32_MAX - 2 * kBN || T + rq.n > INT32_MAX - 2 * kBN)
      return fail(p, GK_ERR_INVALID, "more tokens than 2^31 - 1");
    rq.t0 = (int32_t)T;
    rq.nt_hot = tiles(rq.lp);
    rq.nt_cold = tiles(rq.ctx);
    rq.row = r;
    T += rq.n;
    if (rq.n > 0) {
      const int64_t past = (int64_t)rq.lp + rq.ctx;
      pairs += rq.n * past + (int64_t)rq.n * (rq.n + 1) / 2;
      kept += rq.ctx;
      table += (rq.ctx + c.cold_page_size - 1) / c.cold_page_size;
      if (rq.lp) {
        pl->any_hot = true;
        used.push_back({base, rq.lp});
      }
      if (rq.ctx) pl->any_cold = true;
      pl->max_blocks = std::max(pl->max_blocks, (rq.ctx + c.cold_page_size - 1) / c.cold_page_size);
    }
    pl->reqs.push_back(rq);
  }
  if (pl->any_hot && c.hot_tokens * c.num_layers * Hkv > INT32_MAX)
    return fail(p, GK_ERR_UNSUPPORTED, "HOT pool of more than 2^31 - 1 rows");
  std::sort(used.begin(), used.end());
  used.erase(std::unique(used.begin(), used.end()), used.end());
  for (auto& u : used) kept += u.second;
  pl->tokens = T;
  const int64_t d = c.head_dim, Hq = c.num_q_heads;
  sum.tokens = T;
  sum.flops = 4 * d * Hq * pairs;
  sum.bytes = 4 * T * Hq * d + 4 * T * Hq + 4 * T * Hkv * d + 4 * kept * Hkv * d + 4 * table;

  // ---- neighbouring requests stacked over their HOT prefix ------------------------
  // Worth it where the tiles saved cost more than joining every row of the run: 64 turns of
  // 1-16 tokens behind one prefix of 16384 take 137 us stacked and 647 us apart; turns of 64-600
  // tokens, which fill their own items, stay apart.  Only neighbours: an item's rows are loaded as
  // one box of the packed tokens.
  std::vector<Run> runs;
  std::vector<int32_t> run_of((size_t)B, -1), run_tok((size_t)B, 0);
  for (int32_t r = 0; r < B;) {
    if (base_of[(size_t)r] < 0 || pl->reqs[(size_t)r].lp == 0) { ++r; continue; }
    int32_t e = r, n = 0;
    double apart = 0, joins = 0;
    auto block_us = [&](int32_t tokens) {         // one prefix tile under all blocks of so many tokens
      return (tokens / bt) * kTile2Us + (tokens % bt == 0 ? 0.0 : tokens % bt > tpt ? kTile2Us : kTile1Us);
    };
    for (; e < B && (base_of[(size_t)e] == base_of[(size_t)r] || pl->reqs[(size_t)e].n == 0); ++e) {
      const int32_t ne = pl->reqs[(size_t)e].n;
      run_tok[(size_t)e] = n;
      n += ne;
      apart += block_us(ne);
      joins += ((int64_t)ne * G + 31) / 32;
    }
    const double saved = (apart - block_us(n)) * pl->reqs[(size_t)r].nt_hot;
    if (saved > joins * kJoinUs + (n + bt - 1) / bt * kItemUs) {
      Run run;
      run.rec = (int32_t)pl->reqs.size();
      run.n = n;
      run.blocks = (n + bt - 1) / bt;
      PromptReqDev rq = pl->reqs[(size_t)r];
      rq.n = n;
      rq.ctx = rq.nt_cold = 0;
      pl->reqs.push_back(rq);
      for (int32_t k = r; k < e; ++k)
        if (pl->reqs[(size_t)k].n > 0) {
          run_of[(size_t)k] = (int32_t)runs.size();
          ++sum.stacked_requests;
        }
      runs.push_back(run);
    }
    r = e;
  }

  // ---- blocks of rows and their key tiles (one KV head's worth) --------------------
  std::vector<Shape> shapes;
  for (size_t u = 0; u < runs.size(); ++u) {
    const PromptReqDev& rq = pl->reqs[(size_t)runs[u].rec];
    for (int32_t k = 0; k < runs[u].blocks; ++k) {
      Shape s{runs[u].rec, k * bt, 0, rq.nt_hot, k * bt + tpt < rq.n};
      s.run = (int32_t)u;
      s.run_block = k;
      s.joined = true;
      shapes.push_back(s);
    }
  }
  for (int32_t r = 0; r < B; ++r) {
    const PromptReqDev& rq = pl->reqs[(size_t)r];
    for (int32_t tok0 = 0; tok0 < rq.n; tok0 += bt) {
      const int32_t last = std::min(rq.n, tok0 + bt) - 1;
      const int32_t first = run_of[(size_t)r] >= 0 ? rq.nt_hot : 0;
      Shape s{r, tok0, first, rq.nt_hot + rq.nt_cold + last / kBN + 1 - first, tok0 + tpt < rq.n};
      s.hot_run = run_of[(size_t)r];
      s.hot_tok = run_tok[(size_t)r] + tok0;
      s.joined = s.hot_run >= 0;
      shapes.push_back(s);
    }
  }

  // ---- how many key tiles one item takes -------------------------------------------
  // Whole ranges, or pieces of at most `most` tiles where the balance over the SMs
  // gains more than the join costs (steps with few rows and many keys): the same 64 turns take
  // 137 us in pieces and 195 us whole; one question of 77 tokens, with one tile, stays whole.
  const int num_sms = p->dev.num_sms;
  double work = 0, longest_us = 0;
  int32_t longest = 1;
  for (const Shape& s : shapes) {
    work += Hkv * cost(s, s.ntile);
    longest = std::max(longest, s.ntile);
    longest_us = std::max(longest_us, cost(s, s.ntile));
  }
  const double mean = work / num_sms;
  int32_t best = longest;
  double best_t = 1e300;
  // Two dozen items per SM, none of which stands out, balance by themselves.  With one that does
  // (a single context of 131072 tokens among 456 of 16) whole ranges leave an SM with 1025 tiles where
  // the others have 48: two sizes are tried then, as each takes some 100 ns of host time an item.
  const bool many = shapes.size() * (size_t)Hkv >= 24 * (size_t)num_sms;
  if (!many || longest_us > mean / 8) {
    for (int k = 0; k <= (many ? 2 : 8); ++k) {
      const int32_t most = k == 0 ? longest : std::max(1, (int32_t)(mean / kTile2Us / k));
      if (k > 0 && most >= longest) continue;
      std::vector<double> costs;
      double joined = 0;
      for (const Shape& s : shapes) {
        const int32_t np = pieces_of(s.ntile, most);
        for (int32_t x = 0; x < np; ++x)
          for (int32_t h = 0; h < Hkv; ++h) costs.push_back(cost(s, s.ntile / np + (x < s.ntile % np)));
        if (s.run < 0 && (np > 1 || s.joined))
          joined += (double)Hkv * ((std::min(bt, pl->reqs[(size_t)s.req].n - s.tok0) * G + 31) / 32) * np;
      }
      double t = balance(costs, num_sms, nullptr);
      if (joined > 0) t += kJoinLaunchUs + joined * kJoinUs / num_sms;
      if (t < best_t) {
        best_t = t;
        best = most;
      }
      if (best_t <= mean + kJoinLaunchUs) break;   // pieces add a join to at least this much
    }
  }

  // ---- items, partial states, joins --------------------------------------------------
  std::vector<PromptItemDev> items;
  std::vector<double> costs;
  int64_t entries = 0, part_rows = 0;             // a state has as many rows as its block
  for (const Shape& s : shapes) {                 // the runs come first: their entries are known to the joins
    const int32_t np = pieces_of(s.ntile, best);
    sum.max_pieces = std::max(sum.max_pieces, np);
    const bool parts = np > 1 || s.joined;
    const int32_t rows = std::min(bt, pl->reqs[(size_t)s.req].n - s.tok0) * G;
    for (int32_t h = 0; h < Hkv; ++h) {
      int64_t entry = -1, part_row = -1;
      if (s.run >= 0) {
        Run& run = runs[(size_t)s.run];
        if (s.run_block == 0 && h == 0) {
          run.entry0 = (int32_t)entries;
          run.row0 = part_rows;
          run.pieces = np;
          entries += (int64_t)Hkv * run.blocks * np;
          part_rows += (int64_t)Hkv * run.n * G * np;
        }
        entry = run.entry0 + ((int64_t)h * run.blocks + s.run_block) * np;
        part_row = run.row0 + ((int64_t)h * run.n + s.tok0) * G * np;    // the blocks before are whole
      } else if (parts) {
        entry = entries;
        part_row = part_rows;
        entries += np;
        part_rows += (int64_t)np * rows;
        for (int32_t row = 0; row < rows; row += 32) {
          PromptJoinDev jn{s.req, h, s.tok0, row, (int32_t)part_row, np, 0, 0, s.hot_tok, 0};
          if (s.hot_run >= 0) {
            const Run& run = runs[(size_t)s.hot_run];
            jn.hot0 = (int32_t)(run.row0 + (int64_t)h * run.n * G * run.pieces);
            jn.hot_n = run.pieces;
            jn.hot_len = run.n;
          }
          pl->joins.push_back(jn);
        }
      }
      if (part_rows > INT32_MAX) return fail(p, GK_ERR_INVALID, "too many partial states");
      int32_t tile = s.tile0;
      for (int32_t x = 0; x < np; ++x) {
        const int32_t nt = s.ntile / np + (x < s.ntile % np);
        items.push_back({s.req, h, s.tok0, tile, nt, parts ? (int32_t)entry + x : -1,
                         parts ? (int32_t)(part_row + (int64_t)x * rows) : -1, 0});
        costs.push_back(cost(s, nt));
        tile += nt;
      }
    }
  }
  pl->n_entries = (int32_t)entries;
  pl->part_rows = part_rows;

  // ---- CTA lists ---------------------------------------------------------------------
  const int ctas = (int)std::min<size_t>((size_t)num_sms, items.size());
  if (ctas > 0) {
    std::vector<int32_t> bin;
    balance(costs, ctas, &bin);
    // Within a CTA request by request, the last blocks of each first: what runs side by side on
    // the SMs then reads one request's K and V, and ends with its shortest items.  16 prompts of
    // 1024 tokens take 130 us so, 145 with the longest items of all requests first and 180 with
    // every other CTA's list turned round.
    std::vector<int32_t> order(items.size());
    for (size_t i = 0; i < order.size(); ++i) order[i] = (int32_t)i;
    std::stable_sort(order.begin(), order.end(), [&](int32_t x, int32_t y) {
      return bin[(size_t)x] != bin[(size_t)y] ? bin[(size_t)x] < bin[(size_t)y] : x > y;
    });
    pl->cta_begin.assign((size_t)ctas + 1, 0);
    std::vector<int32_t> load((size_t)ctas, 0);
    for (int32_t i : order) {
      pl->items.push_back(items[(size_t)i]);
      ++pl->cta_begin[(size_t)bin[(size_t)i] + 1];
      load[(size_t)bin[(size_t)i]] += items[(size_t)i].ntile;
    }
    for (int k = 0; k < ctas; ++k) pl->cta_begin[(size_t)k + 1] += pl->cta_begin[(size_t)k];
    sum.max_cta_tiles = *std::max_element(load.begin(), load.end());
  }
  sum.items = (int32_t)items.size();
  sum.ctas = ctas;
  sum.partials = pl->n_entries;
  sum.scratch_bytes = part_rows * (d + 1) * (int64_t)sizeof(float);
  pl->summary = sum;
  return GK_OK;
}

size_t region(size_t* off, size_t bytes) {
  const size_t at = *off;
  *off = (at + bytes + 63) & ~(size_t)63;
  return at;
}

gk_status upload(Pool* p, PromptPlan* pl, void* stream) {
  cudaStream_t st = (cudaStream_t)stream;
  if (pl->any_hot && encode_hot_maps(&p->cfg, pl->hot_maps))
    return fail(p, GK_ERR_CUDA, "encoding the HOT pool's tensor maps failed");
  size_t off = 0;
  pl->off_reqs = region(&off, pl->reqs.size() * sizeof(PromptReqDev));
  pl->off_items = region(&off, pl->items.size() * sizeof(PromptItemDev));
  pl->off_begin = region(&off, pl->cta_begin.size() * sizeof(int32_t));
  pl->off_joins = region(&off, pl->joins.size() * sizeof(PromptJoinDev));
  cudaError_t e;
  if (off > pl->d_bytes) {
    if (pl->d_buf) {
      e = cudaStreamSynchronize(st);
      if (e != cudaSuccess) return cuda_fail(p, e, "cudaStreamSynchronize");
      cudaFree(pl->d_buf);
      cudaFreeHost(pl->h_stage);
      pl->d_buf = pl->h_stage = nullptr;
      pl->d_bytes = 0;
    }
    const size_t cap = off + off / 2;
    e = cudaMalloc(&pl->d_buf, cap);
    if (e != cudaSuccess) return cuda_fail(p, e, "cudaMalloc(prompt plan)");
    e = cudaHostAlloc(&pl->h_stage, cap, cudaHostAllocDefault);
    if (e != cudaSuccess) {
      cudaFree(pl->d_buf);
      pl->d_buf = nullptr;
      return cuda_fail(p, e, "cudaHostAlloc(prompt plan staging)");
    }
    pl->d_bytes = cap;
  } else if (pl->staged) {
    // the previous upload must have left the staging buffer before it is rewritten
    e = cudaEventSynchronize(pl->upload_done);
    if (e != cudaSuccess) return cuda_fail(p, e, "cudaEventSynchronize");
  }
  uint8_t* h = (uint8_t*)pl->h_stage;
  auto put = [&](size_t o, const void* src, size_t bytes) { if (bytes) std::memcpy(h + o, src, bytes); };
  put(pl->off_reqs, pl->reqs.data(), pl->reqs.size() * sizeof(PromptReqDev));
  put(pl->off_items, pl->items.data(), pl->items.size() * sizeof(PromptItemDev));
  put(pl->off_begin, pl->cta_begin.data(), pl->cta_begin.size() * sizeof(int32_t));
  put(pl->off_joins, pl->joins.data(), pl->joins.size() * sizeof(PromptJoinDev));
  e = cudaMemcpyAsync(pl->d_buf, h, off, cudaMemcpyHostToDevice, st);
  if (e != cudaSuccess) return cuda_fail(p, e, "prompt plan upload");
  if (!pl->upload_done) {
    e = cudaEventCreateWithFlags(&pl->upload_done, cudaEventDisableTiming);
    if (e != cudaSuccess) return cuda_fail(p, e, "cudaEventCreate");
  }
  e = cudaEventRecord(pl->upload_done, st);
  if (e != cudaSuccess) return cuda_fail(p, e, "cudaEventRecord");
  pl->staged = true;
  if ((size_t)pl->part_rows > pl->part_cap) {
    if (pl->d_part_o) {
      e = cudaStreamSynchronize(st);
      if (e != cudaSuccess) return cuda_fail(p, e, "cudaStreamSynchronize");
      cudaFree(pl->d_part_o);
      cudaFree(pl->d_part_l);
      pl->d_part_o = pl->d_part_l = nullptr;
      pl->part_cap = 0;
    }
    const size_t cap = (size_t)pl->part_rows + (size_t)pl->part_rows / 4;
    e = cudaMalloc(&pl->d_part_o, cap * (size_t)p->cfg.head_dim * sizeof(float));
    if (e != cudaSuccess) return cuda_fail(p, e, "cudaMalloc(prompt partial outputs)");
    e = cudaMalloc(&pl->d_part_l, cap * sizeof(float));
    if (e != cudaSuccess) {
      cudaFree(pl->d_part_o);
      pl->d_part_o = nullptr;
      return cuda_fail(p, e, "cudaMalloc(prompt partial lse)");
    }
    pl->part_cap = cap;
  }
  pl->uploaded = true;
  return GK_OK;
}

gk_status plan_for(Pool* p, PromptPlan* pl, const gk_prompt_batch* b, void* stream) {
  if (p->has_device) {
    // a captured upload would read the staging buffer of whatever step is planned at its replay
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    const cudaError_t e = cudaStreamIsCapturing((cudaStream_t)stream, &cap);
    if (e != cudaSuccess) return cuda_fail(p, e, "cudaStreamIsCapturing");
    if (cap != cudaStreamCaptureStatusNone)
      return fail(p, GK_ERR_UNSUPPORTED, "a prompt plan cannot be built or updated while the stream is capturing");
  }
  pl->uploaded = false;
  if (p->has_device) {
    gk_status st = ensure_device(p);
    if (st == GK_OK) st = device_is_current(p);
    if (st != GK_OK) return st;
  }
  gk_status st = GK_ERR_INVALID;
  try {
    st = build_host(p, b, pl);
  } catch (const std::exception&) {       // the host tables did not fit in memory
    return fail(p, GK_ERR_INVALID, "out of host memory while planning");
  }
  if (st != GK_OK) return st;
  return p->has_device ? upload(p, pl, stream) : GK_OK;
}

void free_buffers(PromptPlan* pl) {
  if (pl->d_buf) cudaFree(pl->d_buf);
  if (pl->h_stage) cudaFreeHost(pl->h_stage);
  if (pl->d_part_o) cudaFree(pl->d_part_o);
  if (pl->d_part_l) cudaFree(pl->d_part_l);
  if (pl->upload_done) cudaEventDestroy(pl->upload_done);
}

}  // namespace

gk_status device_is_current(Pool* p) {
  int dev = -1;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(p, e, "cudaGetDevice");
  return dev == p->dev.device ? GK_OK : fail(p, GK_ERR_INVALID, "the pool's device is not the current device");
}

}  // namespace gk

extern "C" {

gk_status gk_prompt_plan_build(gk_pool* pool, const gk_prompt_batch* batch, void* stream, gk_prompt_plan** out) {
  if (!pool || !batch || !out) return GK_ERR_INVALID;
  *out = nullptr;
  gk_prompt_plan* pl = new (std::nothrow) gk_prompt_plan;
  if (!pl) return GK_ERR_INVALID;
  gk_status st = gk::plan_for(&pool->impl, &pl->impl, batch, stream);
  if (st != GK_OK) {
    gk::free_buffers(&pl->impl);
    delete pl;
    return st;
  }
  *out = pl;
  return GK_OK;
}

gk_status gk_prompt_plan_update(gk_prompt_plan* plan, const gk_prompt_batch* batch, void* stream) {
  if (!plan || !batch || !plan->impl.pool) return GK_ERR_INVALID;
  return gk::plan_for(plan->impl.pool, &plan->impl, batch, stream);
}

void gk_prompt_plan_destroy(gk_prompt_plan* plan) {
  if (!plan) return;
  gk::free_buffers(&plan->impl);
  delete plan;
}

gk_status gk_prompt_plan_info(const gk_prompt_plan* plan, gk_prompt_plan_summary* out) {
  if (!plan || !out) return GK_ERR_INVALID;
  *out = plan->impl.summary;
  return GK_OK;
}

gk_status gk_prompt_plan_items(const gk_prompt_plan* plan, int32_t* n_ctas, int32_t* n_items, int32_t* begin,
                               int32_t* items) {
  if (!plan || !n_ctas || !n_items) return GK_ERR_INVALID;
  const gk::PromptPlan& pl = plan->impl;
  *n_ctas = pl.cta_begin.empty() ? 0 : (int32_t)pl.cta_begin.size() - 1;
  *n_items = (int32_t)pl.items.size();
  if (begin) std::copy(pl.cta_begin.begin(), pl.cta_begin.end(), begin);
  if (items)
    for (size_t i = 0; i < pl.items.size(); ++i) {
      const gk::PromptItemDev& it = pl.items[i];
      const gk::PromptReqDev& rq = pl.reqs[(size_t)it.req];
      int32_t* o = items + 8 * i;
      o[0] = rq.row;
      o[1] = it.req >= pl.n_requests ? rq.n : 0;
      o[2] = it.head;
      o[3] = it.tok0;
      o[4] = it.tile0;
      o[5] = it.ntile;
      o[6] = it.entry;
      o[7] = rq.nt_hot;
    }
  return GK_OK;
}

gk_status gk_prompt_attn(gk_pool* pool, void* stream, int32_t layer, const gk_prompt_batch* b,
                         const gk_prompt_plan* plan) {
  if (!pool || !b || !plan) return GK_ERR_INVALID;
  gk::Pool* p = &pool->impl;
  const gk::PromptPlan* pl = &plan->impl;
  const gk_pool_config& c = p->cfg;
  if (layer < 0 || layer >= c.num_layers) return gk::fail(p, GK_ERR_INVALID, "layer out of range");
  if (pl->pool != p) return gk::fail(p, GK_ERR_INVALID, "plan belongs to another pool");
  const bool rows = pl->tokens > 0;
  if (rows && (!b->d_q || !b->d_k || !b->d_v || !b->d_out))
    return gk::fail(p, GK_ERR_INVALID, "batch device pointers missing");
  if (pl->any_cold && !b->d_block_table) return gk::fail(p, GK_ERR_INVALID, "block table missing");
  if (pl->any_cold && b->max_blocks < pl->max_blocks)
    return gk::fail(p, GK_ERR_INVALID, "block-table row shorter than the planned contexts");
  for (const void* ptr : {b->d_q, b->d_k, b->d_v, (const void*)b->d_out})
    if (rows && (uintptr_t)ptr % 16 != 0) return gk::fail(p, GK_ERR_INVALID, "q, k, v and out must be 16-byte aligned");
  if (rows && ((uintptr_t)b->d_lse % 4 != 0 || (uintptr_t)b->d_block_table % 4 != 0))
    return gk::fail(p, GK_ERR_INVALID, "lse and the block table must be 4-byte aligned");
  const int64_t q_row = (int64_t)c.num_q_heads * c.head_dim, kv_row = (int64_t)c.num_kv_heads * c.head_dim;
  const int64_t most = (int64_t)1 << 38;          // a tensor map's stride is below 2^40 bytes
  for (auto s : {std::make_pair(b->q_stride, q_row), std::make_pair(b->k_stride, kv_row),
                 std::make_pair(b->v_stride, kv_row), std::make_pair(b->out_stride, q_row)})
    if (s.first != 0 && (s.first < s.second || s.first % 8 != 0 || s.first > most))
      return gk::fail(p, GK_ERR_INVALID, "a token stride must be 0 or a multiple of 8 that holds the token's heads");
  if (!pl->uploaded) return gk::fail(p, GK_ERR_INVALID, "plan has no device tables");
  if (!rows) return GK_OK;
  gk_status st = gk::ensure_device(p);
  if (st == GK_OK) st = gk::device_is_current(p);
  if (st != GK_OK) return st;
  gk::LaunchCommon lc{&p->cfg, p->d_error, p->dev.num_sms};
  int e = gk::launch_prompt(lc, stream, layer, b, pl);
  return e ? gk::cuda_fail(p, e, "prompt attention kernel") : GK_OK;
}

}  // extern "C"
