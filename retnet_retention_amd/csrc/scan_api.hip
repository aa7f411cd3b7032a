// C-ABI host layer of the gated recurrence, the short convolution and the cache of
// parked states: argument validation, workspace carving and launches on the
// caller's stream.
#include "host_checks.hpp"
#include "scan.hpp"
#include "state_cache.hpp"

namespace {

using namespace ret_host;
using ret::tile_count;

constexpr int64_t kMaxTokens = (int64_t)INT32_MAX - 65536;  // room for a tile behind the last token
constexpr int kSmallestTile = 128;                            // tokens of a workgroup where there are many
constexpr int64_t kMaxTileStride = 1 << 22;
constexpr int64_t kMaxThreads = (int64_t)1 << 32;           // of a launch

// Bounds that the sequence calls share; threads: of a launch, for each token tile
// and channel group
ret_status_t check_shape(int32_t batch, int32_t seqlen, int32_t width, int32_t dtype, bool packed, int64_t total,
                         int64_t threads_per_tile) {
  if (batch < 1 || seqlen < 1 || width < 1 || width > ret::kMaxScanWidth) return RET_ERR_SHAPE;
  const int64_t tokens = packed ? total : (int64_t)batch * seqlen;
  if (tokens < 0 || tokens > kMaxTokens) return RET_ERR_SHAPE;
  const int64_t tiles = tile_count(batch, seqlen, packed, total, kSmallestTile);
  if (tiles > INT32_MAX || tiles * ((width + 63) / 64) >= kMaxThreads / threads_per_tile) return RET_ERR_SHAPE;
  if (dtype != RET_F32 && dtype != RET_BF16) return RET_ERR_UNSUPPORTED;
  return RET_OK;
}

// A token stride (0: the width itself) and the bytes its tensor spans.
bool stride_ok(int64_t stride, int32_t width) { return stride == 0 || (stride >= width && stride < (int64_t)1 << 31); }
int64_t stride_of(int64_t stride, int32_t width) { return stride ? stride : width; }
size_t span_bytes(size_t tokens, int64_t stride, int32_t width, size_t size) {
  return tokens ? ((tokens - 1) * (size_t)stride + width) * size : 0;
}

struct Carve {
  char* base;
  size_t used = 0;
  template <typename P>
  void part(P*& p, size_t bytes) {
    p = base ? reinterpret_cast<P*>(base + used) : nullptr;
    used += align_up(bytes);
  }
};

// ------------------------------------------------------------------ recurrence
ret_status_t check_scan(const ret_scan_desc_t* d, bool packed, int64_t total) {
  if (!d) return RET_ERR_NULL;
  const ret_status_t st = check_shape(d->batch, d->seqlen, d->width, d->dtype, packed, total, 1024);
  if (st != RET_OK) return st;
  const int64_t strides[] = {d->x_stride, d->decay_stride, d->gate_stride};
  for (const int64_t s : strides) {
    if (!stride_ok(s, d->width)) return RET_ERR_SHAPE;
    // a tile is addressed with 32 bits from its first row
    if (s >= kMaxTileStride && (packed || d->seqlen > 1)) return RET_ERR_SHAPE;
  }
  return RET_OK;
}

struct ScanSizes {
  size_t tokens, x, decay, gate, o, ddecay, state, weight, kept;
  int64_t tiles, bwd_tiles;
  bool chain, bwd_chain;  // whether tiles hand anything on
};
ScanSizes sizes_of(const ret_scan_desc_t* d, bool packed, int64_t total, bool gates) {
  ScanSizes s;
  const size_t e = elem_size(d->dtype), de = gates ? e : sizeof(float);
  s.tokens = packed ? (size_t)total : (size_t)d->batch * d->seqlen;
  s.x = span_bytes(s.tokens, stride_of(d->x_stride, d->width), d->width, e);
  s.decay = span_bytes(s.tokens, stride_of(d->decay_stride, d->width), d->width, de);
  s.gate = span_bytes(s.tokens, stride_of(d->gate_stride, d->width), d->width, e);
  s.o = s.tokens * d->width * e;
  s.ddecay = s.tokens * d->width * de;
  s.weight = (size_t)d->width * sizeof(float);
  s.state = d->batch * s.weight;
  s.tiles = tile_count(d->batch, d->seqlen, packed, total, ret::kScanTile);
  s.bwd_tiles = tile_count(d->batch, d->seqlen, packed, total, ret::kScanBwdTile);
  s.chain = ret::has_chain(d->seqlen, packed, total, ret::kScanTile);
  s.bwd_chain = ret::has_chain(d->seqlen, packed, total, ret::kScanBwdTile);
  s.kept = s.bwd_tiles * s.weight;
  return s;
}

// control block with the tickets | words handed on | backward: sums of drate | states
// of its own forward. The forward that a backward runs uses the first two before it.
void carve_scan(Carve& c, ret::ScanParams& p, const ScanSizes& s, bool grad, bool own_kept) {
  const bool chain = grad ? s.bwd_chain || (own_kept && s.chain) : s.chain;
  c.part(p.ctrl, ret::kScanCtrlBytes);
  if (chain) c.part(p.hand, (grad ? s.bwd_tiles : s.tiles) * s.weight * 2);
  if (grad) c.part(p.partial, s.kept);
  if (own_kept) c.part(p.kept, s.kept);
}
size_t scan_workspace(const ret_scan_desc_t* d, bool packed, int64_t total, bool grad, bool own_kept) {
  if (check_scan(d, packed, total) != RET_OK) return 0;
  Carve c{nullptr};
  ret::ScanParams p = {};
  carve_scan(c, p, sizes_of(d, packed, total, true), grad, own_kept);
  return c.used;
}

ret::ScanParams params_of(const ret_scan_desc_t* d, const int32_t* cu, const ScanSizes& s, const void* x,
                          const void* decay, const float* rate, const void* gate, const float* state_in) {
  ret::ScanParams p = {};
  p.x = x;
  p.decay = decay;
  p.rate = rate;
  p.gate = gate;
  p.cu = cu;
  p.batch = d->batch;
  p.seqlen = d->seqlen;
  p.width = d->width;
  p.total = (int)s.tokens;
  p.normalize = d->normalize != 0;
  p.x_stride = stride_of(d->x_stride, d->width);
  p.decay_stride = stride_of(d->decay_stride, d->width);
  p.gate_stride = stride_of(d->gate_stride, d->width);
  p.state_in = state_in;
  return p;
}

ret_status_t status_of(hipError_t e) { return e == hipSuccess ? RET_OK : RET_ERR_HIP; }

// ----------------------------------------------------------------- convolution
ret_status_t check_conv(const ret_conv_desc_t* d, bool packed, int64_t total) {
  if (!d) return RET_ERR_NULL;
  const ret_status_t st = check_shape(d->batch, d->seqlen, d->width, d->dtype, packed, total, 1024);
  if (st != RET_OK) return st;
  if (!stride_ok(d->x_stride, d->width)) return RET_ERR_SHAPE;
  if (d->x_stride >= kMaxTileStride && (packed || d->seqlen > 1)) return RET_ERR_SHAPE;  // as check_scan
  if (d->taps < ret::kMinTaps || d->taps > ret::kMaxTaps) return RET_ERR_UNSUPPORTED;
  return RET_OK;
}

struct ConvSizes {
  size_t tokens, x, o, state, weight, bias, partial;
};
ConvSizes sizes_of(const ret_conv_desc_t* d, bool packed, int64_t total) {
  ConvSizes s;
  const size_t e = elem_size(d->dtype);
  s.tokens = packed ? (size_t)total : (size_t)d->batch * d->seqlen;
  s.x = span_bytes(s.tokens, stride_of(d->x_stride, d->width), d->width, e);
  s.o = s.tokens * d->width * e;
  s.state = (size_t)d->batch * (d->taps - 1) * d->width * e;
  s.bias = (size_t)d->width * sizeof(float);
  s.weight = s.bias * d->taps;
  s.partial = (size_t)ret::conv_bwd_blocks(d->batch, d->seqlen, d->width, packed, total) * (s.weight + s.bias);
  return s;
}
void carve_conv(Carve& c, ret::ConvParams& p, const ConvSizes& s, bool grad) {
  c.part(p.ctrl, 2 * sizeof(int32_t));
  if (grad) c.part(p.partial, s.partial);
}
size_t conv_workspace(const ret_conv_desc_t* d, bool packed, int64_t total, bool grad) {
  if (check_conv(d, packed, total) != RET_OK || (!grad && !packed)) return 0;
  Carve c{nullptr};
  ret::ConvParams p = {};
  carve_conv(c, p, sizes_of(d, packed, total), grad);
  return c.used;
}
ret::ConvParams params_of(const ret_conv_desc_t* d, const int32_t* cu, const ConvSizes& s, const void* x,
                          const float* weight, const float* bias, const void* state_in) {
  ret::ConvParams p = {};
  p.x = x;
  p.weight = weight;
  p.bias = bias;
  p.cu = cu;
  p.batch = d->batch;
  p.seqlen = d->seqlen;
  p.width = d->width;
  p.total = (int)s.tokens;
  p.swish = d->swish != 0;
  p.x_stride = stride_of(d->x_stride, d->width);
  p.state_in = state_in;
  return p;
}

// ----------------------------------------------------------- cache of states
ret_status_t check_cache(const ret_state_cache_desc_t* d) {
  if (!d) return RET_ERR_NULL;
  if (d->batch < 1 || d->batch > 65535 || d->values < 1 || d->num_slots < 1 || d->num_slots > INT32_MAX ||
      d->cache_slots < 1 || d->cache_slots > INT32_MAX)
    return RET_ERR_SHAPE;
  // 256 lanes take 1024 values; a launch's threads are counted in 32 bits
  if (d->values > (int64_t)1 << 33 || (d->values + 1023) / 1024 * d->batch >= kMaxThreads / 256) return RET_ERR_SHAPE;
  return RET_OK;
}
ret_status_t cache_call(const ret_state_cache_desc_t* d, const float* state, const int8_t* codes, const float* scales,
                        const int32_t* at, const int32_t* slots, bool write, hipStream_t stream) {
  ret_status_t st = check_cache(d);
  if (st != RET_OK) return st;
  if (!slots && d->num_slots != d->batch) return RET_ERR_SHAPE;
  if (!state || !codes || !scales || !at) return RET_ERR_NULL;
  const int64_t blocks = (d->values + ret::kCacheBlock - 1) / ret::kCacheBlock;
  const size_t list = (size_t)d->batch * sizeof(int32_t);
  const Arg args[] = {{state, (size_t)d->num_slots * d->values * sizeof(float), 16, !write},
                      {codes, (size_t)d->cache_slots * d->values, 16, write},
                      {scales, (size_t)d->cache_slots * blocks * sizeof(float), 16, write},
                      {at, list, 4, false},
                      {slots, list, 4, false}};
  if ((st = check_args(args, 5)) != RET_OK) return st;
  ret::StateCacheParams p = {};
  p.state = const_cast<float*>(state);
  p.codes = const_cast<int8_t*>(codes);
  p.scales = const_cast<float*>(scales);
  p.at = at;
  p.slots = slots;
  p.batch = d->batch;
  p.num_slots = d->num_slots;
  p.cache_slots = d->cache_slots;
  p.values = d->values;
  p.blocks = blocks;
  return status_of(write ? ret::launch_state_cache_write(p, stream) : ret::launch_state_cache_read(p, stream));
}

}  // namespace

extern "C" {

size_t retention_scan_workspace_bytes(const ret_scan_desc_t* desc, int32_t packed, int64_t total_tokens) {
  return scan_workspace(desc, packed != 0, total_tokens, false, false);
}
size_t retention_scan_kept_bytes(const ret_scan_desc_t* desc, int32_t packed, int64_t total_tokens) {
  if (check_scan(desc, packed != 0, total_tokens) != RET_OK) return 0;
  return sizes_of(desc, packed != 0, total_tokens, true).kept;
}

ret_status_t retention_scan_fwd(const ret_scan_desc_t* desc, const int32_t* cu_seqlens, int64_t total_tokens,
                                const void* x, const void* decay, const float* rate, const void* gate, void* o,
                                const float* state_in, float* state_out, float* kept, void* workspace,
                                size_t workspace_bytes, hipStream_t stream) {
  const bool packed = cu_seqlens != nullptr;
  ret_status_t st = check_scan(desc, packed, total_tokens);
  if (st != RET_OK) return st;
  const ScanSizes s = sizes_of(desc, packed, total_tokens, rate != nullptr);
  if (s.tokens && (!x || !decay || !o)) return RET_ERR_NULL;
  const size_t need = scan_workspace(desc, packed, total_tokens, false, false);
  const size_t e = elem_size(desc->dtype), de = rate ? e : sizeof(float);
  const Arg args[] = {{state_in, s.state, 16, false},
                      {state_out, s.state, 16, true},
                      {x, s.x, e, false},
                      {decay, s.decay, de, false},
                      {rate, s.weight, 16, false},
                      {gate, s.gate, e, false},
                      {o, s.o, 16, true},
                      {kept, s.kept, 16, true},
                      {cu_seqlens, ((size_t)desc->batch + 1) * sizeof(int32_t), 4, false},
                      {workspace, need, 16, true}};
  // a sequence's state_in is read before its state_out is written
  if ((st = check_args(args, 9, 0, 1)) != RET_OK) return st;
  if (!workspace || workspace_bytes < need) return RET_ERR_WORKSPACE;
  if ((st = check_args(args, 10, 0, 1)) != RET_OK) return st;
  ret::ScanParams p = params_of(desc, cu_seqlens, s, x, decay, rate, gate, state_in);
  p.o = o;
  p.state_out = state_out;
  Carve c{static_cast<char*>(workspace)};
  carve_scan(c, p, s, false, false);
  p.kept = kept;
  p.tiles = (int)s.tiles;
  return status_of(ret::launch_scan_fwd(p, desc->dtype, stream));
}

size_t retention_scan_bwd_workspace_bytes(const ret_scan_desc_t* desc, int32_t packed, int64_t total_tokens,
                                          int32_t has_kept) {
  return scan_workspace(desc, packed != 0, total_tokens, true, has_kept == 0);
}

ret_status_t retention_scan_bwd(const ret_scan_desc_t* desc, const int32_t* cu_seqlens, int64_t total_tokens,
                                const void* x, const void* decay, const float* rate, const void* gate,
                                const void* dout, const float* state_in, const float* d_state_out, const float* kept,
                                void* dx, void* ddecay, float* drate, void* dgate, float* d_state_in, void* workspace,
                                size_t workspace_bytes, hipStream_t stream) {
  const bool packed = cu_seqlens != nullptr;
  ret_status_t st = check_scan(desc, packed, total_tokens);
  if (st != RET_OK) return st;
  const ScanSizes s = sizes_of(desc, packed, total_tokens, rate != nullptr);
  if (s.tokens && (!x || !decay || !dout || !dx || !ddecay || (gate == nullptr) != (dgate == nullptr)))
    return RET_ERR_NULL;
  if ((rate == nullptr) != (drate == nullptr) || (state_in == nullptr) != (d_state_in == nullptr)) return RET_ERR_NULL;
  const size_t need = scan_workspace(desc, packed, total_tokens, true, kept == nullptr);
  const size_t e = elem_size(desc->dtype), de = rate ? e : sizeof(float);
  const Arg args[] = {{x, s.x, e, false},
                      {decay, s.decay, de, false},
                      {rate, s.weight, 16, false},
                      {gate, s.gate, e, false},
                      {dout, s.o, 16, false},
                      {state_in, s.state, 16, false},
                      {d_state_out, s.state, 16, false},
                      {kept, s.kept, 16, false},
                      {cu_seqlens, ((size_t)desc->batch + 1) * sizeof(int32_t), 4, false},
                      {dx, s.o, 16, true},
                      {ddecay, s.ddecay, 16, true},
                      {drate, s.weight, 16, true},
                      {dgate, s.o, 16, true},
                      {d_state_in, s.state, 16, true},
                      {workspace, need, 16, true}};
  if ((st = check_args(args, 14)) != RET_OK) return st;
  if (!workspace || workspace_bytes < need) return RET_ERR_WORKSPACE;
  if ((st = check_args(args, 15)) != RET_OK) return st;
  ret::ScanParams p = params_of(desc, cu_seqlens, s, x, decay, rate, gate, state_in);
  p.dout = dout;
  p.d_state_out = d_state_out;
  p.d_state_in = d_state_in;
  p.dx = dx;
  p.ddecay = ddecay;
  p.dgate = dgate;
  p.drate = drate;
  Carve c{static_cast<char*>(workspace)};
  carve_scan(c, p, s, true, kept == nullptr);
  uint64_t* hand = p.hand;
  if (!kept) {  // the forward once more, for the states alone
    p.tiles = (int)s.tiles;
    p.hand = s.chain ? hand : nullptr;
    if (ret::launch_scan_fwd(p, desc->dtype, stream) != hipSuccess) return RET_ERR_HIP;
    p.keep_error = true;
  } else {
    p.kept = const_cast<float*>(kept);
  }
  p.tiles = (int)s.bwd_tiles;
  p.hand = s.bwd_chain ? hand : nullptr;
  return status_of(ret::launch_scan_bwd(p, desc->dtype, stream));
}

ret_status_t retention_scan_step(const ret_scan_desc_t* desc, const void* x, const void* decay, const float* rate,
                                 const void* gate, void* o, float* state, const int32_t* slots, int64_t num_slots,
                                 hipStream_t stream) {
  ret_status_t st = check_scan(desc, false, 0);
  if (st != RET_OK) return st;
  if (desc->seqlen != 1 || desc->batch > 65535) return RET_ERR_SHAPE;
  if (num_slots < 1 || num_slots > INT32_MAX || (!slots && num_slots != desc->batch)) return RET_ERR_SHAPE;
  if (!x || !decay || !o || !state) return RET_ERR_NULL;
  const ScanSizes s = sizes_of(desc, false, 0, rate != nullptr);
  const size_t e = elem_size(desc->dtype), de = rate ? e : sizeof(float);
  const Arg args[] = {{x, s.x, e, false},
                      {decay, s.decay, de, false},
                      {rate, s.weight, 16, false},
                      {gate, s.gate, e, false},
                      {slots, (size_t)desc->batch * sizeof(int32_t), 4, false},
                      {o, s.o, 16, true},
                      {state, num_slots * s.weight, 16, true}};
  if ((st = check_args(args, 7)) != RET_OK) return st;
  ret::ScanStepParams p = {};
  p.x = x;
  p.decay = decay;
  p.rate = rate;
  p.gate = gate;
  p.o = o;
  p.state = state;
  p.slots = slots;
  p.batch = desc->batch;
  p.width = desc->width;
  p.num_slots = (int)num_slots;
  p.normalize = desc->normalize != 0;
  p.x_stride = stride_of(desc->x_stride, desc->width);
  p.decay_stride = stride_of(desc->decay_stride, desc->width);
  p.gate_stride = stride_of(desc->gate_stride, desc->width);
  return status_of(ret::launch_scan_step(p, desc->dtype, stream));
}

size_t retention_conv_workspace_bytes(const ret_conv_desc_t* desc, int32_t packed, int64_t total_tokens) {
  return conv_workspace(desc, packed != 0, total_tokens, false);
}

ret_status_t retention_conv_fwd(const ret_conv_desc_t* desc, const int32_t* cu_seqlens, int64_t total_tokens,
                                const void* x, const float* weight, const float* bias, void* o, const void* state_in,
                                void* state_out, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const bool packed = cu_seqlens != nullptr;
  ret_status_t st = check_conv(desc, packed, total_tokens);
  if (st != RET_OK) return st;
  const ConvSizes s = sizes_of(desc, packed, total_tokens);
  if (!weight || (s.tokens && (!x || !o))) return RET_ERR_NULL;
  const size_t need = conv_workspace(desc, packed, total_tokens, false);
  const Arg args[] = {{state_in, s.state, 16, false},
                      {state_out, s.state, 16, true},
                      {x, s.x, elem_size(desc->dtype), false},
                      {weight, s.weight, 16, false},
                      {bias, s.bias, 16, false},
                      {o, s.o, 16, true},
                      {cu_seqlens, ((size_t)desc->batch + 1) * sizeof(int32_t), 4, false},
                      {workspace, need, 16, true}};
  // the wave that reads a part of state_in writes that part of state_out afterwards
  if ((st = check_args(args, 7, 0, 1)) != RET_OK) return st;
  if (need && (!workspace || workspace_bytes < need)) return RET_ERR_WORKSPACE;
  if ((st = check_args(args, need ? 8 : 7, 0, 1)) != RET_OK) return st;
  ret::ConvParams p = params_of(desc, cu_seqlens, s, x, weight, bias, state_in);
  p.o = o;
  p.state_out = state_out;
  if (need) {
    Carve c{static_cast<char*>(workspace)};
    carve_conv(c, p, s, false);
  }
  return status_of(ret::launch_conv_fwd(p, desc->taps, desc->dtype, stream));
}

size_t retention_conv_bwd_workspace_bytes(const ret_conv_desc_t* desc, int32_t packed, int64_t total_tokens) {
  return conv_workspace(desc, packed != 0, total_tokens, true);
}

ret_status_t retention_conv_bwd(const ret_conv_desc_t* desc, const int32_t* cu_seqlens, int64_t total_tokens,
                                const void* x, const float* weight, const float* bias, const void* dout,
                                const void* state_in, const void* d_state_out, void* dx, float* dweight, float* dbias,
                                void* d_state_in, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const bool packed = cu_seqlens != nullptr;
  ret_status_t st = check_conv(desc, packed, total_tokens);
  if (st != RET_OK) return st;
  const ConvSizes s = sizes_of(desc, packed, total_tokens);
  if (!weight || !dweight || (s.tokens && (!x || !dout || !dx))) return RET_ERR_NULL;
  if ((bias == nullptr) != (dbias == nullptr) || (state_in == nullptr) != (d_state_in == nullptr)) return RET_ERR_NULL;
  const size_t need = conv_workspace(desc, packed, total_tokens, true);
  const Arg args[] = {{x, s.x, elem_size(desc->dtype), false},
                      {weight, s.weight, 16, false},
                      {bias, s.bias, 16, false},
                      {dout, s.o, 16, false},
                      {state_in, s.state, 16, false},
                      {d_state_out, s.state, 16, false},
                      {cu_seqlens, ((size_t)desc->batch + 1) * sizeof(int32_t), 4, false},
                      {dx, s.o, 16, true},
                      {dweight, s.weight, 16, true},
                      {dbias, s.bias, 16, true},
                      {d_state_in, s.state, 16, true},
                      {workspace, need, 16, true}};
  if ((st = check_args(args, 11)) != RET_OK) return st;
  if (!workspace || workspace_bytes < need) return RET_ERR_WORKSPACE;
  if ((st = check_args(args, 12)) != RET_OK) return st;
  ret::ConvParams p = params_of(desc, cu_seqlens, s, x, weight, bias, state_in);
  p.dout = dout;
  p.d_state_out = d_state_out;
  p.d_state_in = d_state_in;
  p.dx = dx;
  p.dweight = dweight;
  p.dbias = dbias;
  Carve c{static_cast<char*>(workspace)};
  carve_conv(c, p, s, true);
  return status_of(ret::launch_conv_bwd(p, desc->taps, desc->dtype, stream));
}

ret_status_t retention_conv_step(const ret_conv_desc_t* desc, const void* x, const float* weight, const float* bias,
                                 void* o, void* state, const int32_t* slots, int64_t num_slots, hipStream_t stream) {
  ret_status_t st = check_conv(desc, false, 0);
  if (st != RET_OK) return st;
  if (desc->seqlen != 1 || desc->batch > 65535) return RET_ERR_SHAPE;
  if (num_slots < 1 || num_slots > INT32_MAX || (!slots && num_slots != desc->batch)) return RET_ERR_SHAPE;
  if (!x || !weight || !o || !state) return RET_ERR_NULL;
  const ConvSizes s = sizes_of(desc, false, 0);
  const Arg args[] = {{x, s.x, elem_size(desc->dtype), false},
                      {weight, s.weight, 16, false},
                      {bias, s.bias, 16, false},
                      {slots, (size_t)desc->batch * sizeof(int32_t), 4, false},
                      {o, s.o, 16, true},
                      {state, s.state / desc->batch * num_slots, 16, true}};
  if ((st = check_args(args, 6)) != RET_OK) return st;
  ret::ConvStepParams p = {};
  p.x = x;
  p.weight = weight;
  p.bias = bias;
  p.o = o;
  p.state = state;
  p.slots = slots;
  p.batch = desc->batch;
  p.width = desc->width;
  p.num_slots = (int)num_slots;
  p.swish = desc->swish != 0;
  p.x_stride = stride_of(desc->x_stride, desc->width);
  return status_of(ret::launch_conv_step(p, desc->taps, desc->dtype, stream));
}

ret_status_t retention_state_cache_write(const ret_state_cache_desc_t* desc, const float* state, int8_t* codes,
                                         float* scales, const int32_t* cache_slots, const int32_t* slots,
                                         hipStream_t stream) {
  return cache_call(desc, state, codes, scales, cache_slots, slots, true, stream);
}
ret_status_t retention_state_cache_read(const ret_state_cache_desc_t* desc, const int8_t* codes, const float* scales,
                                        float* state, const int32_t* cache_slots, const int32_t* slots,
                                        hipStream_t stream) {
  return cache_call(desc, state, codes, scales, cache_slots, slots, false, stream);
}

}  // extern "C"
