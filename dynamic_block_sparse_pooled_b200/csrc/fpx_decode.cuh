// fpx_decode.cuh -- what the decode kernels share: the problem as they see it, the work line that
// plan lays out and the split of it among workers, and the layout of partial results.
//
// Decode attention of a batch is a set of segments: (rows that share keys) x (a range of cached
// keys) for one KV head.  A request's own part gives segments of its q_len x group rows over
// [prefix, ctx); a group's shared prompt gives segments of the rows of all its requests over the
// prompt.  All segments of a launch stand end to end on one line of units (a key tile is one, and a
// segment has a few more for what it costs in itself), and worker w of NW takes the units
// [w W / NW, (w + 1) W / NW): every worker has the same work whatever the lengths are (NW <= W: with
// fewer units than workers some stay idle).  A segment cut by worker borders leaves one partial (running maximum, sum,
// unnormalised O; 32 bits) per worker; partial slot = segment index + worker index, which differs
// for any two pieces since each step along the line moves one of the two.  A last kernel joins
// each row's partials in slot order, so a result does not depend on timing.
#pragma once

#include <cuda.h>

#include "fpx_common.cuh"
#include "fpx_rule.cuh"

namespace fpx {
namespace decode {

struct DecodeDesc {
  int num_seqs, q_len, hq, hkv, group, d, page, log2_page;
  int pages_per_seq, num_pages, num_groups, tokens;  // tokens = num_seqs * q_len
  float scale;
  const float* k_scale;
  const float* v_scale;
  const int32_t* ctx;
  const int32_t* table;
  const int32_t* group_ptr;
  const int32_t* prefix_pages;
  RuleDesc rule;
};

// A request's own keys, or a group's shared ones.
struct __align__(16) Owner {
  int k0, k1;      // keys [k0, k1), k0 a multiple of min(page, 32)
  int tok0, ntok;  // query tokens
  int row;         // block-table row
  int line;        // first unit on the line
  int seg;         // first segment
  int nrt;         // row tiles per KV head
};

// One launch over a line.  owners has n + 1 entries; the last one's line is the total.
struct Line {
  Owner* owners;
  int n;     // owners
  int rt;    // rows of a row tile
  int tile;  // keys of a tile
  int nw;    // workers
  int pad;   // units of the line in front of a segment's tiles
  int rps;   // rows stored per partial slot
  // 0: a row tile is rt consecutive rows (token x group + head).  Else the 128-row form: tiles of
  // tpt whole tokens, a segment has a pair of them, tile i of the pair at rows 128 i of its slot; a
  // segment with one tile leaves two partials of it, at rows 0 and 128.
  int tpt;
  float* part_o;    // [slots][rps][d]
  float2* part_ml;  // [slots][rps]: maximum (log2 units), sum
};

// Workers that take part: none is left without a unit, so every slot between the first and the
// last worker of a segment is written.
__device__ __forceinline__ int64_t active_workers(const Line& l, int64_t total) {
  return total < l.nw ? total : l.nw;
}
__device__ __forceinline__ int64_t line_begin(int64_t w, int64_t total, int64_t nw) {
  return w * total / nw;
}
// The worker whose range holds unit x: the largest w with w * total / nw <= x.
__device__ __forceinline__ int worker_of(int64_t x, int64_t total, int64_t nw) {
  return static_cast<int>(((x + 1) * nw - 1) / total);
}

__device__ __forceinline__ int tiles_of(const Owner& w, int tile) {
  return w.k1 > w.k0 ? (w.k1 - w.k0 + tile - 1) / tile : 0;
}

__device__ __forceinline__ Owner load_owner(const Owner* o) {
  const int4* p = reinterpret_cast<const int4*>(o);
  const int4 a = p[0], b = p[1];
  return {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
}

// Units of a segment on the line: its tiles, behind `pad` units that stand for what a worker spends
// on a segment whatever its length (rows of Q, the partial).
__device__ __forceinline__ int units_of(const Owner& w, const Line& l) {
  const int n = tiles_of(w, l.tile);
  return n > 0 ? n + l.pad : 0;
}

// A worker's walk over its stretch of the line, one piece (consecutive tiles of one segment) at a
// time.  All lanes of a warp walk alike.
struct Walk {
  const Line* line;
  Owner w;
  int o, j, u;     // owner, segment of the owner, unit of the segment
  int left;        // units of the stretch from (o, j, u) on
  int t0, cnt;     // the piece: tiles t0 .. t0 + cnt - 1, cnt > 0
  __device__ __forceinline__ void enter(const Line& l, int x0, int x1) {
    line = &l;
    left = x1 - x0;
    if (left == 0) return;
    int lo = 0, hi = l.n - 1;  // the last owner with line <= x0: it has units, as x0 < total
    while (lo < hi) {
      const int mid = lo + ((hi - lo + 1) >> 1);
      if (l.owners[mid].line <= x0) lo = mid;
      else hi = mid - 1;
    }
    o = lo;
    w = load_owner(l.owners + o);
    const int per = units_of(w, l), rem = x0 - w.line;
    j = rem / per;
    u = rem - j * per;
  }
  // On to the next piece; false at the end of the stretch.
  __device__ __forceinline__ bool next(int hkv) {
    while (left > 0) {
      const int per = units_of(w, *line);
      if (u >= per) {
        u = 0;
        if (++j >= w.nrt * hkv || per == 0) {
          j = 0;
          if (++o >= line->n) return false;
          w = load_owner(line->owners + o);
        }
        continue;
      }
      const int take = min(left, per - u);
      const int a = max(u - line->pad, 0), b = max(u + take - line->pad, 0);
      u += take;
      left -= take;
      if (b > a) {
        t0 = a;
        cnt = b - a;
        return true;
      }
    }
    return false;
  }
};

// Where a query row stands and what it sees.
struct RowPos {
  int i;
  KeySpan span;
};
__device__ __forceinline__ RowPos row_pos(const DecodeDesc& p, int token) {
  const int s = token / p.q_len;
  const int most = p.pages_per_seq << p.log2_page;
  const int ctx = min(max(p.ctx[s], 0), most);
  RowPos r;
  r.i = ctx - p.q_len + (token - s * p.q_len);
  r.span = rule_span(p.rule, token, r.i, ctx);
  if (r.i < 0) r.span = {0, -1};
  return r;
}

// The shared prompts on the tensor cores of the fifth generation (fpx_decode_sm100.cu).
bool tc_supported(const DecodeDesc& p, fpx_dtype dt);
void tc_line(const DecodeDesc& p, Line* l);  // rt, tile, rps and tpt of the 128-row form
cudaError_t launch_tc(const DecodeDesc& p, const Line& line, const void* q, const void* kc,
                      const void* vc, StatusBlock* st, cudaStream_t s, bool* encode_failed);

}  // namespace decode

cudaError_t launch_decode(const decode::DecodeDesc& p, fpx_dtype dt, const void* q, const void* kc,
                          const void* vc, void* o, float* lse, void* ws, StatusBlock* st,
                          cudaStream_t s, bool* encode_failed);
size_t decode_workspace(const decode::DecodeDesc& p, fpx_dtype dt);
bool decode_fits(const decode::DecodeDesc& p, fpx_dtype dt);

}  // namespace fpx
