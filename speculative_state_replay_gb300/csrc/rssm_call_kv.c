/* rssm_call_kv.c -- the fast path of rssm_call.c for the calls of attention layers and of the sampler. */
#include "rssm_call.h"

static PyObject *kv_append(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
  TAKE(15)
  const rssm_kv_cache *c = P(0);
  const int32_t layer = I32(1);
  const void *k = P(2), *v = P(4);
  const int64_t ks = I64(3), vs = I64(5);
  const int32_t *pages = P(6);
  const int64_t ps = I64(7);
  const int32_t max_pages = I32(8);
  const int32_t *lengths = P(9), *cu = P(10);
  const int32_t batch = I32(11), T = I32(12);
  const int64_t tokens = I64(13);
  void *stream = P(14);
  GIVE(rssm_kv_append(c, layer, k, ks, v, vs, pages, ps, max_pages, lengths, cu, batch, T, tokens, stream));
}

static PyObject *kv_read(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
  TAKE(15)
  const rssm_kv_cache *c = P(0);
  const int32_t layer = I32(1);
  const int32_t *pages = P(2);
  const int64_t ps = I64(3);
  const int32_t max_pages = I32(4);
  const int32_t *starts = P(5), *cu = P(6);
  const int32_t batch = I32(7);
  const int64_t tokens = I64(8);
  const int32_t dtype = I32(9);
  void *k = P(10), *v = P(12);
  const int64_t ks = I64(11), vs = I64(13);
  void *stream = P(14);
  GIVE(rssm_kv_read(c, layer, pages, ps, max_pages, starts, cu, batch, tokens, dtype, k, ks, v, vs, stream));
}

static PyObject *tree_attention(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
  TAKE(20)
  const rssm_kv_cache *c = P(0);
  const int32_t layer = I32(1);
  const void *q = P(2);
  const int64_t qs = I64(3);
  const int32_t heads = I32(4);
  const float scale = F32(5);
  const int32_t *pages = P(6);
  const int64_t ps = I64(7);
  const int32_t max_pages = I32(8);
  const int32_t *lengths = P(9), *parents = P(10), *cu = P(11);
  const int32_t batch = I32(12), T = I32(13);
  const int64_t tokens = I64(14);
  void *out = P(15);
  const int64_t os = I64(16);
  void *scratch = P(17);
  const int64_t bytes = I64(18);
  void *stream = P(19);
  GIVE(rssm_tree_attention(c, layer, q, qs, heads, scale, pages, ps, max_pages, lengths, parents, cu, batch, T, tokens, out, os,
                           scratch, (size_t)bytes, stream));
}

static PyObject *tree_accept(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
  TAKE(17)
  const rssm_kv_cache *c = P(0);
  const int32_t *pages = P(1);
  const int64_t ps = I64(2);
  const int32_t max_pages = I32(3);
  const int32_t *lengths = P(4), *tokens = P(5), *parents = P(6), *drawn = P(7), *cu = P(8);
  const int32_t batch = I32(9), T = I32(10);
  const int64_t ntok = I64(11);
  int32_t *accepted = P(12), *next = P(13), *path = P(14);
  uint32_t *word = P(15);
  void *stream = P(16);
  GIVE(rssm_tree_accept(c, pages, ps, max_pages, lengths, tokens, parents, drawn, cu, batch, T, ntok, accepted, next, path, word,
                        stream));
}

static PyObject *logits(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
  TAKE(31)
  rssm_logits_args a;
  a.logits = P(0);
  a.logits_stride = I64(1);
  a.logits_dtype = I32(2);
  a.out = P(3);
  a.out_stride = I64(4);
  a.out_dtype = I32(5);
  a.vocab = I32(6);
  a.batch = I32(7);
  a.T = I32(8);
  a.probs = I32(9);
  a.ntok = I64(10);
  a.cu_seqlens = P(11);
  a.temperature = P(12);
  a.repetition = P(13);
  a.presence = P(14);
  a.frequency = P(15);
  a.history = P(16);
  a.history_stride = I64(17);
  a.history_max = I32(18);
  a.history_len = P(19);
  a.prompt_len = P(20);
  a.tokens = P(21);
  a.parents = P(22);
  a.bias_start = P(23);
  a.bias_id = P(24);
  a.bias_value = P(25);
  a.biases = I64(26);
  a.mask = P(27);
  a.mask_stride = I64(28);
  a.error_word = P(29);
  void *stream = P(30);
  GIVE(rssm_logits(&a, stream));
}

static PyMethodDef methods[] = {
    {"rssm_kv_append", (PyCFunction)(void (*)(void))kv_append, METH_FASTCALL, NULL},
    {"rssm_kv_read", (PyCFunction)(void (*)(void))kv_read, METH_FASTCALL, NULL},
    {"rssm_tree_attention", (PyCFunction)(void (*)(void))tree_attention, METH_FASTCALL, NULL},
    {"rssm_tree_accept", (PyCFunction)(void (*)(void))tree_accept, METH_FASTCALL, NULL},
    {"rssm_logits", (PyCFunction)(void (*)(void))logits, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_call_kv", "C calls into librssm with checked arguments", -1,
                                    methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__call_kv(void) { return PyModule_Create(&module); }
