"""The paged cache calls refuse what they cannot do before anything is launched, and the
index arithmetic they share with the kernels is checked exhaustively (CPU only)."""
import ctypes as ct
import os
import re
import struct
import subprocess

import pytest

import train_step_b200 as tsb

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x7F0000001000  # an address that is never read: every call below is refused on the host

CONFIG, TOO_LONG, BATCH = -1, -3, -5


@pytest.fixture(scope="module", autouse=True)
def built():
    from train_step_b200 import build
    build.build()


def cache(**kw):
    f = dict(k=A, v=A, page_stride=16 * 2 * 64, row_stride=2 * 64, head_stride=64, page_table=A, table_stride=8,
             status=None, dtype=tsb.BF16, n_pages=100, page_size=16, max_pages=8, n_seqs=3, n_kv_heads=2, head_dim=64)
    f.update(kw)
    return tsb._PagedKV(**f)


def append(kv, **kw):
    f = dict(k=A, ldk=128, v=A, ldv=128, q=A, ldq=256, q_out=A, ldqo=256, nh=4, N=3, positions=A, seqs=A, cos_sin=A,
             n_positions=128, rot=64, pairs=0)
    f.update(kw)
    rows = tsb._PAGED_ROWS.pack(*(f[n] or 0 for n in (
        "k", "v", "q", "q_out", "ldk", "ldv", "ldq", "ldqo", "positions", "seqs", "cos_sin", "N", "nh", "n_positions",
        "rot", "pairs")))
    return tsb.lib().gpt2_op_paged_kv_append(kv if kv is None else ct.byref(kv), rows, None)


def attend(kv, **kw):
    f = dict(q=A, ldq=256, nh=4, lens=A, scale=0.125, window=0, sinks=0, out=A, ldo=256, lse=A, ws=A, ws_bytes=1 << 40)
    f.update(kw)
    query = tsb._PAGED_QUERY.pack(*(f[n] or 0 for n in (
        "q", "out", "lse", "lens", "ws", "ws_bytes", "ldq", "ldo", "nh", "window", "sinks", "scale")))
    return tsb.lib().gpt2_op_paged_attention(kv if kv is None else ct.byref(kv), query, None)


BAD_CACHES = [
    (dict(k=None), CONFIG), (dict(v=None), CONFIG), (dict(page_table=None), CONFIG), (dict(k=A + 8), CONFIG),
    (dict(v=A + 2), CONFIG), (dict(page_table=A + 2), CONFIG), (dict(status=A + 1), CONFIG), (dict(dtype=7), CONFIG),
    (dict(head_dim=48), CONFIG), (dict(head_dim=0), CONFIG), (dict(head_dim=256), CONFIG), (dict(n_pages=0), CONFIG),
    (dict(max_pages=0), CONFIG), (dict(n_kv_heads=0), CONFIG), (dict(n_kv_heads=2048), CONFIG),
    (dict(n_seqs=-1), CONFIG), (dict(n_seqs=4097), BATCH), (dict(page_size=24), CONFIG), (dict(page_size=0), CONFIG),
    (dict(page_size=8192), CONFIG), (dict(table_stride=7), CONFIG), (dict(page_stride=2052), CONFIG),
    (dict(row_stride=-128), CONFIG), (dict(head_stride=4), CONFIG),
    (dict(max_pages=1 << 20, table_stride=1 << 20, page_size=2048), TOO_LONG),
    (dict(max_pages=1 << 20, table_stride=1 << 20, page_size=512, n_seqs=33), TOO_LONG),
]


@pytest.mark.parametrize("change,code", BAD_CACHES)
def test_a_bad_cache_is_refused_by_both_calls(change, code):
    assert append(cache(**change)) == code
    assert attend(cache(**change)) == code
    assert b"paged cache" in tsb.lib().gpt2_op_last_error()


def test_a_null_cache_is_refused():
    assert append(None) == CONFIG and attend(None) == CONFIG
    kv = cache()
    assert tsb.lib().gpt2_op_paged_kv_append(ct.byref(kv), None, None) == CONFIG
    assert tsb.lib().gpt2_op_paged_attention(ct.byref(kv), None, None) == CONFIG
    assert tsb.lib().gpt2_op_paged_status(None, None) == CONFIG
    assert tsb.lib().gpt2_op_paged_status(ct.byref(cache()), None) == CONFIG  # no status word


@pytest.mark.parametrize("change,code", [
    (dict(k=None), CONFIG), (dict(v=None), CONFIG), (dict(k=A + 8), CONFIG), (dict(ldk=120), CONFIG),
    (dict(ldv=132), CONFIG), (dict(q=None), CONFIG), (dict(q_out=None), CONFIG), (dict(nh=0), CONFIG),
    (dict(nh=-1), CONFIG), (dict(nh=5000, ldq=320000, ldqo=320000), CONFIG), (dict(ldq=248), CONFIG),
    (dict(ldqo=260), CONFIG), (dict(q_out=A + 4), CONFIG), (dict(N=-1), CONFIG), (dict(positions=None), CONFIG),
    (dict(seqs=None, N=4), BATCH), (dict(N=1 << 29), BATCH), (dict(rot=8), CONFIG), (dict(rot=80), CONFIG), (dict(rot=-16), CONFIG),
    (dict(positions=A + 2), CONFIG), (dict(seqs=A + 1), CONFIG), (dict(cos_sin=None), CONFIG), (dict(cos_sin=A + 4), CONFIG), (dict(n_positions=0), CONFIG),
])
def test_append_refuses(change, code):
    assert append(cache(), **change) == code
    assert b"paged_kv_append" in tsb.lib().gpt2_op_last_error()


@pytest.mark.parametrize("strides", [
    dict(head_stride=0), dict(head_stride=56), dict(row_stride=64), dict(page_stride=0), dict(page_stride=1984),
    dict(row_stride=0), dict(head_stride=2048, row_stride=64, page_stride=2048), dict(page_stride=(1 << 63) - 8)])
def test_append_refuses_a_cache_whose_heads_overlap(strides):
    kv = cache(**strides)
    assert append(kv) == CONFIG and b"overlap" in tsb.lib().gpt2_op_last_error()
    assert append(kv, N=0) == CONFIG


@pytest.mark.parametrize("strides", [
    dict(head_stride=0, n_kv_heads=1), dict(row_stride=0, page_size=1, max_pages=8), dict(page_stride=0, n_pages=1),
    dict(head_stride=1024, row_stride=64), dict(page_stride=64, head_stride=6400, row_stride=12800),
    dict(page_stride=4096)])
def test_append_takes_any_order_of_the_cache_and_dimensions_of_one(strides):
    assert append(cache(**strides), N=0) == 0


def test_append_of_no_rows_does_nothing():
    assert append(cache(), N=0) == 0
    assert append(cache(), N=0, positions=None) == 0


@pytest.mark.parametrize("change,code", [
    (dict(q=None), CONFIG), (dict(out=None), CONFIG), (dict(q=A + 8), CONFIG), (dict(ldq=248), CONFIG),
    (dict(ldo=252), CONFIG), (dict(nh=0), CONFIG), (dict(nh=3), CONFIG), (dict(nh=4098), CONFIG),
    (dict(lens=None), CONFIG), (dict(lens=A + 2), CONFIG), (dict(lse=A + 3), CONFIG), (dict(scale=2e38), CONFIG), (dict(scale=0.0), CONFIG), (dict(scale=-1.0), CONFIG),
    (dict(scale=float("nan")), CONFIG), (dict(scale=float("inf")), CONFIG), (dict(window=-1), CONFIG),
    (dict(sinks=-1), CONFIG), (dict(ws=None), CONFIG), (dict(ws=A + 8), CONFIG), (dict(ws_bytes=0), CONFIG),
])
def test_attention_refuses(change, code):
    assert attend(cache(), **change) == code
    assert b"paged_attention" in tsb.lib().gpt2_op_last_error()


def test_attention_of_no_sequences_does_nothing():
    assert attend(cache(n_seqs=0)) == 0
    assert attend(cache(n_seqs=0, page_table=None), lens=None, q=None) == 0


def test_workspace_size():
    f = tsb.lib().gpt2_paged_attention_ws_bytes
    assert f(3, 4, 2, 64) > 0 and f(0, 4, 2, 64) > 0 and f(4096, 128, 1, 128) > 0
    for bad in ((-1, 4, 2, 64), (4097, 4, 2, 64), (3, 5, 2, 64), (3, 0, 2, 64), (3, 4, 0, 64), (3, 4, 2, 0),
                (3, 4, 2, 48)):
        assert f(*bad) == 0


def test_packed_structs_are_those_of_the_header(tmp_path):
    src = tmp_path / "layout.c"
    names = ["k", "v", "q", "q_out", "ldk", "ldv", "ldq", "ldqo", "positions", "seqs", "f32_cos_sin", "n_rows",
             "n_q_heads", "n_positions", "rot_dim", "interleaved"]
    query = ["q", "out", "f32_lse", "seq_lens", "ws", "ws_bytes", "ldq", "ldo", "n_q_heads", "window", "sinks", "scale"]
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "gpt2.h"\nint main(void) {\n' + "".join(
        f'printf("%zu ", offsetof({t}, {n}));\n' for t, ns in (("gpt2_paged_rows", names), ("gpt2_paged_query", query),
        ("gpt2_paged_kv", [f[0] for f in tsb._PagedKV._fields_])) for n in ns) + "return 0; }\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I" + os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]

    def offsets(fmt):
        codes = "".join(c * int(n or 1) for n, c in re.findall(r"(\d*)([a-zA-Z])", fmt))
        return [struct.calcsize("@" + codes[:i] + "0" + codes[i]) for i in range(len(codes))]
    assert got == (offsets(tsb._PAGED_ROWS.format) + offsets(tsb._PAGED_QUERY.format)
                   + [getattr(tsb._PagedKV, f[0]).offset for f in tsb._PagedKV._fields_])


INDEX_CHECK = r"""
#include <cstdlib>
#include <set>
#include <vector>
#include "paged_index.cuh"
using namespace g2;
int main() {
  for (int len = 0; len < 70; ++len)
    for (int window = 0; window < 75; ++window)
      for (int sinks = 0; sinks < 75; ++sinks) {
        std::set<int> want, got;
        for (int j = 0; j < len; ++j)
          if (window == 0 || j >= len - window || j < sinks) want.insert(j);
        const PagedVisible v = paged_visible(len, window, sinks);
        int last = -1;
        for (int t = 0; t < v.tiles; ++t) {
          const int pos = paged_tile_pos(v, t);
          const uint32_t mask = paged_tile_mask(v, pos);
          if (pos % PAT_TILE || pos <= last || mask == 0 || mask > 0xffff) return 1;
          last = pos;
          for (int i = 0; i < PAT_TILE; ++i)
            if (mask >> i & 1) got.insert(pos + i);
        }
        if (got != want) return 2;
      }
  // the extremes do not overflow
  const int big = 1 << 30, most = 0x7fffffff;
  if (paged_visible(big, most, most).tiles != big / 16 || paged_visible(big, 1, most).tiles != big / 16) return 3;
  const PagedVisible one = paged_visible(big, 1, 0);
  if (one.tiles != 1 || paged_tile_pos(one, 0) != big - 16 || paged_tile_mask(one, big - 16) != 0x8000) return 4;
  if (paged_div(7, 2) != 3 || paged_div(1LL << 40, 3) != (1LL << 40) / 3 || paged_div(0xffffffffLL, 1) != 0xffffffffLL) return 13;
  int bad = 0;
  if (paged_length(5, 10, &bad) != 5 || paged_length(10, 10, &bad) != 10 || bad) return 5;
  if (paged_length(11, 10, &bad) != 10 || !bad) return 6;
  bad = 0;
  if (paged_length(-3, 10, &bad) != 0 || !bad) return 7;

  for (int d : {1, 2, 3, 7, 48, 144, 1000, 65537, 0x7fffffff})
    for (int64_t x : {0LL, 1LL, 2LL, 143LL, 144LL, 1LL << 20, 0x7ffffffeLL, 0x7fffffffLL})
      for (int64_t k : {-1LL, 0LL, 1LL}) {
        const int64_t y = x / d * d + k;  // around every multiple
        if (y >= 0 && y <= 0x7fffffff && paged_div_by((int)y, d, 0xffffffffu / d) != y / d) return 14;
        if (paged_div_by((int)x, d, 0xffffffffu / d) != x / d) return 15;
      }

  // every worker's walk over its share, one after the other, is the whole order
  srand(1);
  for (int trial = 0; trial < 3000; ++trial) {
    const int n_seqs = 1 + rand() % 9, items = 1 + rand() % 5, workers = 1 + rand() % 40;
    std::vector<int> before(n_seqs + 1, 0);
    for (int b = 0; b < n_seqs; ++b) before[b + 1] = before[b] + (rand() % 3 ? rand() % 14 : 0);
    const int64_t total = (int64_t)before[n_seqs] * items, share = paged_share(total, workers, 0xffffffffu / workers);
    if (share < 1 || share * workers < total) return 8;
    int64_t u = 0;
    int seq = -1, item = items - 1, tile = 0, tiles = 1;  // the walk that is expected
    for (int w = 0; w < workers; ++w) {
      const int64_t a = w * share, e = a + share < total ? a + share : total;
      if (a >= e) continue;
      int at = 0;  // the sequence of tile a
      while ((int64_t)before[at + 1] * items <= a) ++at;
      PagedCursor c = paged_place(before.data(), at, items, a);
      for (int64_t i = a; i < e; ++i, ++u) {
        if (i > a) {
          const int was = c.seq;
          if (paged_next(c, before.data(), items) != (c.seq != was)) return 9;
        }
        if (u == 0 || ++tile >= tiles) {
          tile = 0;
          if (++item >= items) {
            item = 0;
            do ++seq;
            while (before[seq + 1] == before[seq]);
            tiles = before[seq + 1] - before[seq];
          }
        }
        if (c.seq != seq || c.item != item || c.tile != tile || c.tiles != tiles) return 10;
      }
    }
    if (u != total) return 11;
  }
  return 0;
}
"""


def test_index_arithmetic(tmp_path):
    src = tmp_path / "check.cpp"
    src.write_text(INDEX_CHECK)
    exe = tmp_path / "check"
    subprocess.run(["g++", "-O1", "-std=c++17", "-x", "c++", "-I" + os.path.join(ROOT, "train_step_b200", "csrc"),
                    str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0


def test_rotation_table_of_far_positions():
    import numpy as np
    n, rot = 200001, 48
    got = tsb.rotation_table(n, rot, base=500000.0, device="cpu").numpy()
    assert got.shape == (n, rot) and got.dtype == np.float32
    for t in (0, 1, 4095, 131071, 200000):
        for i in (0, 1, 11, 23):
            angle = np.longdouble(t) * np.longdouble(500000.0) ** (-np.longdouble(2 * i) / rot)
            # one rounding to fp32, and the angle's own in float64 (t of them at most 2^18, 53 bits)
            for x, want in ((got[t, i], np.cos(angle)), (got[t, rot // 2 + i], np.sin(angle))):
                assert abs(float(x) - float(want)) <= 2.0 ** -24 * abs(float(want)) + 2.0 ** -33
    assert tsb.rotation_table(5, 0, device="cpu").shape == (5, 0)


def test_binding_refuses_what_is_not_on_a_gpu():
    import torch
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        tsb.PagedKV(k, k.clone(), torch.zeros(2, 2, dtype=torch.int32))


GUARD_CHECK = r"""
#include <dlfcn.h>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <new>
#include "gpt2.h"
// the library's allocations come here, and fail when `full`
static bool full = false;
void* operator new(std::size_t n) {
  void* p = full ? nullptr : std::malloc(n);
  if (!p) throw std::bad_alloc();
  return p;
}
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, std::size_t) noexcept { std::free(p); }
int main(int, char** argv) {
  void* lib = dlopen(argv[1], RTLD_NOW);
  if (!lib) return std::printf("%s\n", dlerror()), 1;
  auto append = (decltype(&gpt2_op_paged_kv_append))dlsym(lib, "gpt2_op_paged_kv_append");
  auto attend = (decltype(&gpt2_op_paged_attention))dlsym(lib, "gpt2_op_paged_attention");
  auto status = (decltype(&gpt2_op_paged_status))dlsym(lib, "gpt2_op_paged_status");
  auto error = (decltype(&gpt2_op_last_error))dlsym(lib, "gpt2_op_last_error");
  // in each case the message of the refusal, then the same without memory for it
  for (int i = 0; i < 3; ++i) {
    auto call = [&] { return i == 0 ? append(nullptr, nullptr, nullptr) : i == 1 ? attend(nullptr, nullptr, nullptr)
                                                                                  : status(nullptr, nullptr); };
    full = true;  // first, while no string has memory from before
    const int none = call();
    full = false;
    if (i < 2 && (none != GPT2_ERR_OOM || !std::strstr(error(), "memory"))) return 10 + i;
    if (i == 2 && none != GPT2_ERR_OOM && none != GPT2_ERR_CONFIG) return 12;
    if (call() != GPT2_ERR_CONFIG || !std::strstr(error(), "paged")) return 20 + i;
    full = true;
    const int again = call();
    full = false;
    if (again == GPT2_ERR_OOM ? !std::strstr(error(), "memory") : again != GPT2_ERR_CONFIG) return 30 + i;
  }
  return 0;
}
"""


def test_host_memory_that_runs_out_is_reported_as_that(tmp_path):
    # no exception leaves the library, and the message is that of the failure, not of an earlier one
    src, exe = tmp_path / "guard.cpp", tmp_path / "guard"
    src.write_text(GUARD_CHECK)
    subprocess.run(["g++", "-O1", "-std=c++17", "-rdynamic", "-I" + os.path.join(ROOT, "include"), str(src), "-o",
                    str(exe), "-ldl"], check=True)
    got = subprocess.run([str(exe), tsb.LIB_PATH], capture_output=True, text=True, timeout=60)
    assert got.returncode == 0, (got.returncode, got.stdout, got.stderr)


def test_status_refuses_a_misaligned_word():
    for at in (1, 2, 3):
        assert tsb.lib().gpt2_op_paged_status(ct.byref(cache(status=A + at)), None) == CONFIG
        assert b"aligned" in tsb.lib().gpt2_op_last_error()


@pytest.mark.parametrize("change", [
    dict(q_out=A, ldqo=264), dict(q_out=A, ldqo=512), dict(q_out=A, ldq=264), dict(q_out=A + 16), dict(q_out=A + 512),
    dict(q=A + 512), dict(q=A + 1040, ldq=512, q_out=A, ldqo=520), dict(q_out=A, ldqo=768, ldq=768, k=A + 496, ldk=768),
    dict(q=A + 8192, ldq=512, k=A + 512, ldk=512, v=A + 784, ldv=512, q_out=A, ldqo=512, N=2)])
def test_append_refuses_overlapping_query_rows(change):
    # (elements are 2 bytes; a row of 4 query heads has 512, one of 2 key heads 256)
    f = dict(k=A + (1 << 20), v=A + (2 << 20))
    f.update(change)
    assert append(cache(), **f) == CONFIG
    assert b"q_out" in tsb.lib().gpt2_op_last_error()


@pytest.mark.parametrize("dtype,ld", [(tsb.FP32, 1 << 62), (tsb.BF16, 1 << 62), (tsb.FP32, (1 << 63) - 64), (tsb.BF16, (1 << 63) - 64)])
def test_append_checks_row_strides_of_any_size(dtype, ld):
    # strides whose bytes do not fit 64 bits
    f = dict(k=A + (1 << 20), v=A + (2 << 20), ldq=ld, ldqo=ld)
    assert append(cache(dtype=dtype), **f, q_out=A + 16) == CONFIG
    assert b"q_out" in tsb.lib().gpt2_op_last_error()
    assert append(cache(dtype=dtype), **f, q_out=A + 16, N=1) == CONFIG


APART_CHECK = r"""
#include <set>
#include "paged_index.cuh"
using namespace g2;
int main() {
  for (int n = 1; n <= 4; ++n)
    for (int wa = 1; wa <= 3; ++wa)
      for (int wb = 1; wb <= 3; ++wb)
        for (int lda = wa; lda <= 8; ++lda)
          for (int ldb = wb; ldb <= 8; ++ldb)
            for (int d = -36; d <= 36; ++d) {
              bool apart = true, in_place = true;
              for (int i = 0; i < n; ++i)
                for (int j = 0; j < n; ++j) {
                  const int a = i * lda, b = d + j * ldb;
                  if (a + wa <= b || b + wb <= a) continue;
                  apart = false;
                  if (i != j || a != b || wa != wb) in_place = false;
                }
              if (paged_rows_apart(lda, wa, d, ldb, wb, n, false) != apart) return 1;
              if (paged_rows_apart(lda, wa, d, ldb, wb, n, true) != in_place) return 2;
            }
  const int64_t far = INT64_MAX / 2;  // strides that overflow 64 bits when they are multiplied out
  if (!paged_rows_apart(far, 64, 64, far, 64, 1 << 20, false) || paged_rows_apart(far, 64, 32, far, 64, 1 << 20, true)) return 3;
  return 0;
}
"""


def test_overlap_of_rows(tmp_path):
    src, exe = tmp_path / "apart.cpp", tmp_path / "apart"
    src.write_text(APART_CHECK)
    subprocess.run(["g++", "-O1", "-std=c++17", "-I" + os.path.join(ROOT, "train_step_b200", "csrc"), str(src), "-o",
                    str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0
