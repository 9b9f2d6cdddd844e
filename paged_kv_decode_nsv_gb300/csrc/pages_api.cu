// Host side of the page operators: argument checks and launches.

#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "pages.cuh"

namespace nsv {
namespace {

constexpr int64_t kMaxBlockVecs = 1 << 24;  // 256 MiB, 32768 KV heads of 128 bf16 dims

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// The parameters that follow from the shape and the device.
int page_params(const nsv_shape* s, PageParams* p) {
  const int64_t vecs =
      (int64_t)s->num_kv_heads * kBlock * s->head_dim * (s->dtype == NSV_F32 ? 4 : 2) / 16;
  if (vecs > kMaxBlockVecs) return NSV_ERR_SHAPE;
  DeviceInfo d;
  const int rc = device_info(&d);
  if (rc) return rc;
  p->status = d.status;
  p->num_sms = d.num_sms;
  p->num_blocks = s->num_blocks;
  p->rows = s->rows;
  p->max_blocks = s->max_blocks;
  p->block_vecs = (int)vecs;
  p->units_per_block = page_units(p->block_vecs);
  return NSV_OK;
}

// Null and alignment checks of one call's arguments.
struct Args {
  bool null = false, misaligned = false;
  void need(const void* p, uintptr_t a) {
    null |= !p;
    misaligned |= !aligned(p, a);
  }
  int code() const { return null ? NSV_ERR_NULLPTR : misaligned ? NSV_ERR_ALIGN : NSV_OK; }
};

int check_ws(const nsv_shape* s, void* ws, size_t bytes) {
  return ws && aligned(ws, 256) && bytes >= page_ws_bytes(s->rows, s->num_blocks)
             ? NSV_OK
             : NSV_ERR_WORKSPACE;
}

}  // namespace
}  // namespace nsv

using namespace nsv;

extern "C" {

NSV_API int nsv_pages_workspace(const nsv_shape* shape, int64_t* bytes) {
  if (!bytes) return NSV_ERR_NULLPTR;
  const int rc = check_shape(shape);
  if (rc) return rc;
  *bytes = (int64_t)page_ws_bytes(shape->rows, shape->num_blocks);
  return NSV_OK;
}

NSV_API int nsv_blocks_copy(const nsv_shape* shape, int32_t count, const int32_t* src,
                            const int32_t* dst, void* k_pool, void* v_pool, cudaStream_t stream) {
  int rc = check_shape(shape);
  if (rc) return rc;
  if (count < 0) return NSV_ERR_SHAPE;
  if (count == 0) return NSV_OK;
  Args a;
  a.need(src, 4), a.need(dst, 4), a.need(k_pool, 16), a.need(v_pool, 16);
  if ((rc = a.code()) != NSV_OK) return rc;
  PageParams p;
  memset(&p, 0, sizeof p);
  if ((rc = page_params(shape, &p)) != NSV_OK) return rc;
  p.count = count;
  p.parents = src;
  p.children = dst;
  p.k_pool = k_pool;
  p.v_pool = v_pool;
  return launch_blocks_copy(p, stream) == cudaSuccess ? NSV_OK : cuda_fail();
}

NSV_API int nsv_rows_fork(const nsv_shape* shape, int32_t count, const int32_t* parents,
                          const int32_t* children, int32_t* block_tables, int32_t* context_lens,
                          int32_t* block_refs, void* k_pool, void* v_pool, void* workspace,
                          size_t workspace_bytes, cudaStream_t stream) {
  int rc = check_shape(shape);
  if (rc) return rc;
  if (count < 0 || count > shape->rows) return NSV_ERR_SHAPE;
  if (count == 0) return NSV_OK;
  Args a;
  a.need(parents, 4), a.need(children, 4), a.need(block_tables, 4), a.need(context_lens, 4);
  a.need(block_refs, 4), a.need(k_pool, 16), a.need(v_pool, 16);
  if ((rc = a.code()) != NSV_OK) return rc;
  if ((rc = check_ws(shape, workspace, workspace_bytes)) != NSV_OK) return rc;
  PageParams p;
  memset(&p, 0, sizeof p);
  if ((rc = page_params(shape, &p)) != NSV_OK) return rc;
  p.count = count;
  p.parents = parents;
  p.children = children;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.refs = block_refs;
  p.k_pool = k_pool;
  p.v_pool = v_pool;
  p.ws = static_cast<int32_t*>(workspace);
  return launch_rows_fork(p, stream) == cudaSuccess ? NSV_OK : cuda_fail();
}

NSV_API int nsv_rows_extend(const nsv_shape* shape, int64_t tokens, const int32_t* chunk_starts,
                            int32_t* block_tables, int32_t* context_lens, int32_t* block_refs,
                            int64_t* write_slots, void* workspace, size_t workspace_bytes,
                            cudaStream_t stream) {
  int rc = check_shape(shape);
  if (rc) return rc;
  if (tokens < 0 || tokens >= (int64_t(1) << 30)) return NSV_ERR_SHAPE;
  if (shape->rows == 0 || tokens == 0) return NSV_OK;
  Args a;
  a.need(chunk_starts, 4), a.need(block_tables, 4), a.need(context_lens, 4);
  a.need(block_refs, 4), a.need(write_slots, 8);
  if ((rc = a.code()) != NSV_OK) return rc;
  if ((rc = check_ws(shape, workspace, workspace_bytes)) != NSV_OK) return rc;
  PageParams p;
  memset(&p, 0, sizeof p);
  if ((rc = page_params(shape, &p)) != NSV_OK) return rc;
  p.tokens = tokens;
  p.chunk_starts = chunk_starts;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.refs = block_refs;
  p.write_slots = write_slots;
  p.ws = static_cast<int32_t*>(workspace);
  return launch_rows_extend(p, stream) == cudaSuccess ? NSV_OK : cuda_fail();
}

NSV_API int nsv_rows_free(const nsv_shape* shape, int32_t count, const int32_t* rows_list,
                          int32_t* block_tables, int32_t* context_lens, int32_t* block_refs,
                          cudaStream_t stream) {
  int rc = check_shape(shape);
  if (rc) return rc;
  if (count < 0) return NSV_ERR_SHAPE;
  if (shape->rows == 0 || count == 0) return NSV_OK;
  Args a;
  a.need(rows_list, 4), a.need(block_tables, 4), a.need(context_lens, 4), a.need(block_refs, 4);
  if ((rc = a.code()) != NSV_OK) return rc;
  PageParams p;
  memset(&p, 0, sizeof p);
  if ((rc = page_params(shape, &p)) != NSV_OK) return rc;
  p.count = count;
  p.parents = rows_list;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.refs = block_refs;
  return launch_rows_free(p, stream) == cudaSuccess ? NSV_OK : cuda_fail();
}

NSV_API int nsv_blocks_compact(const nsv_shape* shape, int32_t* block_tables,
                               const int32_t* context_lens, int32_t* block_refs, void* k_pool,
                               void* v_pool, void* workspace, size_t workspace_bytes,
                               cudaStream_t stream) {
  int rc = check_shape(shape);
  if (rc) return rc;
  Args a;
  a.need(block_refs, 4), a.need(k_pool, 16), a.need(v_pool, 16);
  if (shape->rows > 0) a.need(block_tables, 4), a.need(context_lens, 4);
  if ((rc = a.code()) != NSV_OK) return rc;
  if ((rc = check_ws(shape, workspace, workspace_bytes)) != NSV_OK) return rc;
  PageParams p;
  memset(&p, 0, sizeof p);
  if ((rc = page_params(shape, &p)) != NSV_OK) return rc;
  p.block_tables = block_tables;
  p.context_lens = const_cast<int32_t*>(context_lens);
  p.refs = block_refs;
  p.k_pool = k_pool;
  p.v_pool = v_pool;
  p.ws = static_cast<int32_t*>(workspace);
  return launch_blocks_compact(p, stream) == cudaSuccess ? NSV_OK : cuda_fail();
}

}  // extern "C"
