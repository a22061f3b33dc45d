// Arguments of the page-assignment launch (host and device side).
#pragma once

#include "common.cuh"

namespace kvq {

struct PagesMeta {  // per sequence, from the scan
  int64_t cu, take0, ret0;  // tokens, pages taken and pages returned before it
  int32_t held, len;        // before the call
  int32_t take, ret;        // its own pages
  int32_t granted, pad;
};
static_assert(sizeof(PagesMeta) == 48, "workspace layout");

struct PagesHead {
  int64_t head, n_tok, n_taken;
};

struct PagesParams {
  int32_t* table;     // [batch][max_pages]
  int32_t* held;      // [batch]
  int32_t* free_ids;  // ring of n_pages ids
  int64_t* ring;      // first free entry, free entries
  int64_t n_pages;
  int max_pages, span, span_shift;
  const int32_t* len;
  const int32_t* n_new;
  int batch;
  int64_t n_slots;
  int32_t* cu;
  int64_t* slots;
  int32_t* pos;  // may be null
  uint32_t* status;
  PagesHead* head;
  PagesMeta* meta;
};

size_t pages_workspace_bytes(int batch);
cudaError_t launch_pages_assign(PagesParams p, void* ws, cudaStream_t st);

}  // namespace kvq
