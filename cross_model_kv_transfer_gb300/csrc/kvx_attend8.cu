// kvx_attend8.cu -- the calls of attention over the 8-bit paged cache, kvx_attend8 and
// kvx_attend8_shared: checks, workspaces, and which kernels a call takes.
#include <cmath>

#include "kvx_attend8.cuh"

namespace {

// A pass of a call whose requests share prefixes: over the prefixes (`all`) or over the
// requests' own slots (`before`).
struct Pass {
  kvx8::Requests req;
  kvx8::Sharing share;
  bool shared;
  float2 *stats;             // of the prefixes: written in their pass
  int parts;                 // in place of `before` and `stats`: what the prefixes leave in parts
  void *part_bytes;
};

kvx_status check(const kvx_attend8_args *a) {
  if (!a) return KVX_ERR_INVALID_ARG;
  const kvx_cache8 &c = a->cache;
  if (const kvx_status st = check_cache8(c)) return st;
  if ((a->dtype != KVX_F32 && a->dtype != KVX_BF16) || a->num_requests < 1 || a->ntok < 0 ||
      a->ntok > INT32_MAX || (!a->cu_seqlens && a->ntok != a->num_requests) || a->max_new < 1 ||
      a->max_len < 0 || a->max_len > INT32_MAX - 1024 || !a->lens || !std::isfinite(a->scale) || a->q_heads < 1 ||
      a->q_heads > 65535 || a->q_heads % c.heads)
    return KVX_ERR_INVALID_ARG;
  if (a->weights && a->weights_stride < a->max_len) return KVX_ERR_INVALID_ARG;
  if (a->weights && a->num_requests > 65535) return KVX_ERR_UNSUPPORTED;
  // the rows of one request and KV head are counted in 32 bits
  if ((int64_t)(a->q_heads / c.heads) * most_new(a) > INT32_MAX - 1024) return KVX_ERR_UNSUPPORTED;
  return KVX_OK;
}

// Enqueue a checked call, or a pass of one.
kvx_status enqueue(const kvx_attend8_args *a, const Pass &pass, cudaStream_t s) {
  const kvx_cache8 &c = a->cache;
  const int size = a->dtype == KVX_BF16 ? 2 : 4;
  AttendParams p;
  p.k = (const uint8_t *)c.k_codes;
  p.v = (const uint8_t *)c.v_codes;
  p.ks = c.k_scale;
  p.vs = c.v_scale;
  p.q = a->q;
  p.out = a->out;
  p.qt = a->q_token_stride;
  p.qh = a->q_head_stride;
  p.ot = a->out_token_stride;
  p.oh = a->out_head_stride;
  p.table = c.block_table;
  p.lens = a->lens;
  p.lse = a->lse;
  p.weights = a->weights;
  p.stats = pass.stats;
  p.status = a->status;
  p.req = pass.req;
  p.share = pass.share;
  p.num_blocks = (int)c.num_blocks;
  // with k = ceil(log2 bs), 2^(31 + k) / bs rounded up is off by less than 2^k / bs
  // a unit, so the quotient is exact below 2^31
  int k = 0;
  while (1 << k < c.block_size) ++k;
  p.bs_shift = 31 + k;
  p.bs_mul = (uint32_t)(((uint64_t)1 << (31 + k)) / c.block_size + 1);
  p.wstride = a->weights_stride;
  p.H = c.heads;
  p.Hq = a->q_heads;
  p.G = a->q_heads / c.heads;
  p.d = c.head_dim;
  p.bs = c.block_size;
  p.max_blocks = c.max_blocks_per_req;
  p.max_len = a->max_len;
  p.max_new = most_new(a);
  p.bf16 = size == 2 && !pass.share.all;    // what a prefix gives stays in fp32
  p.c = a->scale * kLog2e;
  char *ws = (char *)a->workspace;
  if (pass.parts || (pass.share.before && kvx_attend8_own_supports(a)))
    return kvx_attend8_own_launch(a, p, pass.parts, pass.part_bytes, pass.share.all, s);
  if (kvx_attend8_tc_supports(a)) return (pass.shared ? kvx_attend8_tc_launch_shared : kvx_attend8_tc_launch)(a, p, ws, s);
  return (pass.shared ? kvx_attend8_split_launch_shared : kvx_attend8_split_launch)(a, p, ws, s);
}

size_t least_bytes(const kvx_attend8_args *a) {
  return kvx_attend8_tc_supports(a) ? kvx_attend8_tc_least_bytes(a) : kvx_attend8_split_least_bytes(a);
}

// The two passes of a call whose requests share prefixes, as calls of their own, and what
// they leave beside the workspace of the larger one.
struct Shared {
  kvx_attend8_args before, own;
  int parts;                 // 0: one result for each row of the first pass
  size_t out, stats, bytes;
};
kvx_status shared_of(const kvx_attend8_shared_args *a, Shared &s) {
  if (!a) return KVX_ERR_INVALID_ARG;
  if (const kvx_status st = check(&a->own)) return st;
  if (a->own.weights || !a->prefix_table || !aligned_to(a->prefix_table, 4) || !a->prefix_lens || !aligned_to(a->prefix_lens, 4) ||
      !aligned_to(a->groups, 4) || a->max_prefix_blocks < 1 ||
      a->num_prefixes < 1 || (!a->groups && a->num_prefixes != 1) || a->max_group < 1)
    return KVX_ERR_INVALID_ARG;
  s.own = s.before = a->own;
  kvx_attend8_args &b = s.before;
  b.cache.block_table = a->prefix_table;
  b.cache.max_blocks_per_req = a->max_prefix_blocks;
  b.lens = a->prefix_lens;
  b.max_len = a->max_prefix;
  b.num_requests = a->num_prefixes;
  b.cu_seqlens = a->prefix_lens;      // any table: the pass has its own requests
  const int64_t members = a->max_group < a->own.num_requests ? a->max_group : a->own.num_requests;
  const int64_t most = members * (a->own.cu_seqlens ? most_new(&a->own) : 1);
  b.max_new = (int32_t)(most < INT32_MAX ? most : INT32_MAX);
  if (const kvx_status st = check(&b)) return st;
  const auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t one = least_bytes(&b), two = least_bytes(&s.own), rows = (size_t)a->own.ntok * a->own.q_heads;
  s.out = up(one > two ? one : two);
  s.stats = s.out + up(rows * a->own.cache.head_dim * sizeof(float));
  s.bytes = s.stats + up(rows * sizeof(float2));
  // parts lie behind the head, and there is room for those of smaller calls
  const size_t room = kWorkspaceHead + kvx_attend8_parts_bytes(&b);
  s.bytes = s.bytes > room ? s.bytes : room;
  s.parts = kvx_attend8_own_supports(&s.own) ? kvx_attend8_parts(&b) : 0;
  return KVX_OK;
}

bool usable(const kvx_attend8_args *a, size_t least) {
  const int size = a->dtype == KVX_BF16 ? 2 : 4;
  return a->q && a->out && aligned_to(a->q, size) && aligned_to(a->out, size) && a->workspace &&
         aligned_to(a->workspace, 256) && a->workspace_bytes >= least;
}

}  // namespace

extern "C" size_t kvx_attend8_workspace_bytes(const kvx_attend8_args *a) {
  if (check(a) != KVX_OK) return 0;
  return kvx_attend8_tc_supports(a) ? kvx_attend8_tc_workspace_bytes(a) : kvx_attend8_split_workspace_bytes(a);
}

extern "C" kvx_status kvx_attend8(const kvx_attend8_args *a, void *stream) {
  if (const kvx_status st = check(a)) return st;
  if (a->ntok == 0) return KVX_OK;
  if (!usable(a, least_bytes(a))) return KVX_ERR_INVALID_ARG;
  if (a->weights && a->out == a->q) return KVX_ERR_INVALID_ARG;   // scores may be formed again
  Pass pass = {};
  pass.req = {a->cu_seqlens, a->num_requests, a->ntok};
  return enqueue(a, pass, (cudaStream_t)stream);
}

extern "C" size_t kvx_attend8_shared_workspace_bytes(const kvx_attend8_shared_args *a) {
  Shared s;
  return shared_of(a, s) == KVX_OK ? s.bytes : 0;
}

// Two passes: each prefix against the queries of all requests that share it, as one
// request's, and the requests' own slots, whose results are joined with the first pass's
// where they are written.  A prefix is read once for up to 256 rows of its group (8 where the
// slots go in parts, 8 to 32 in the split form) and not once a request, and its products have as
// many: what they cost is that of a prompt of as many tokens.
extern "C" kvx_status kvx_attend8_shared(const kvx_attend8_shared_args *a, void *stream) {
  Shared s;
  if (const kvx_status st = shared_of(a, s)) return st;
  const kvx_attend8_args &own = s.own;
  if (own.ntok == 0) return KVX_OK;
  if (!usable(&own, s.bytes)) return KVX_ERR_INVALID_ARG;
  char *ws = (char *)own.workspace;
  kvx_attend8_args &before = s.before;
  before.out = ws + s.out;
  before.out_token_stride = (int64_t)own.q_heads * own.cache.head_dim;
  before.out_head_stride = own.cache.head_dim;
  before.lse = nullptr;
  Pass pass = {};
  pass.shared = true;
  pass.parts = s.parts;
  pass.part_bytes = ws + kWorkspaceHead;
  pass.stats = (float2 *)(ws + s.stats);
  pass.req = {own.cu_seqlens, a->num_prefixes, own.ntok};
  pass.share.of = a->groups;
  pass.share.inner = own.num_requests;
  pass.share.count = a->num_prefixes;
  pass.share.most = before.max_new;
  pass.share.whole = !a->groups;
  pass.share.all = 1;
  if (const kvx_status st = enqueue(&before, pass, (cudaStream_t)stream)) return st;
  pass.req = {own.cu_seqlens, own.num_requests, own.ntok};
  pass.share.all = 0;
  pass.share.before = (const float *)(ws + s.out);
  pass.share.before_stats = pass.stats;
  pass.stats = nullptr;
  return enqueue(&own, pass, (cudaStream_t)stream);
}
