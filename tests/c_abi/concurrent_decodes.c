/* Paged decodes issued by several host threads at the same time (see tests/test_gpu_paged_threads.py): each
 * thread issues its job's call over and over and counts the statuses other than COWA_OK. */
#include <pthread.h>

#include "cowa.h"

typedef cowa_status (*decode_fn)(const cowa_pattern*, int, int, int, int, const void*, cowa_tensor, cowa_tensor,
                                 cowa_page_table, const int32_t*, void*, float*, void*, size_t, void*);
typedef cowa_status (*decode_fp8_fn)(const cowa_pattern*, int, int, int, int, const void*, cowa_tensor, cowa_tensor,
                                     float, float, cowa_page_table, const int32_t*, void*, float*, void*, size_t, void*);

typedef struct {
  decode_fn decode;         /* the one that is not NULL is called */
  decode_fp8_fn decode_fp8;
  const cowa_pattern* pat;
  const void* q;
  const int32_t* pos;
  void* o;
  float* lse;
  void* ws;
  size_t ws_bytes;
  void* stream;
  cowa_tensor k, v;
  cowa_page_table table;
  int B, Hq, Hkv, d;
  int calls, bad;
} job;

static void* work(void* x) {
  job* j = (job*)x;
  int i;
  for (i = 0; i < j->calls; ++i) {
    cowa_status s = j->decode ? j->decode(j->pat, j->B, j->Hq, j->Hkv, j->d, j->q, j->k, j->v, j->table, j->pos, j->o,
                                          j->lse, j->ws, j->ws_bytes, j->stream)
                              : j->decode_fp8(j->pat, j->B, j->Hq, j->Hkv, j->d, j->q, j->k, j->v, 0.015625f, 0.015625f,
                                              j->table, j->pos, j->o, j->lse, j->ws, j->ws_bytes, j->stream);
    if (s != COWA_OK) ++j->bad;
  }
  return NULL;
}

/* 0, or 1 if a thread could not be started (n <= 16) */
int run_jobs(job* jobs, int n) {
  pthread_t t[16];
  int i, started = 0;
  while (started < n && pthread_create(&t[started], NULL, work, &jobs[started]) == 0) ++started;
  for (i = 0; i < started; ++i) pthread_join(t[i], NULL);
  return started < n;
}
