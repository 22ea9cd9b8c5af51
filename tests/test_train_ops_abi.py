"""Host-side tests of include/train_ops.h: the library exports what the header
declares, a C99 client links every entry point, and bad arguments are refused
before anything touches a GPU."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import optimizer_step_gb300 as og
from optimizer_step_gb300 import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "train_ops.h")


def declared_symbols():
    text = open(HEADER).read()
    return sorted(set(re.findall(r"LAMB_API\s+[\w\s\*]+?\b(train_\w+)\s*\(", text)))


def test_header_binding_and_library_name_the_same_entry_points():
    assert declared_symbols() == sorted(_lib.TRAIN_EXPORTS)
    out = subprocess.run(["nm", "-D", "--defined-only", og.library_path()], capture_output=True,
                         text=True, check=True).stdout
    exported = {ln.split()[-1] for ln in out.splitlines() if " T " in ln}
    assert {s for s in exported if s.startswith("train")} == set(declared_symbols())


def test_a_c99_program_links_and_runs(tmp_path):
    names = declared_symbols()
    src = tmp_path / "client.c"
    src.write_text("#include <stdio.h>\n#include \"train_ops.h\"\n"
                   "typedef void (*entry_point)(void);\n"
                   "static const entry_point points[] = {"
                   + ", ".join("(entry_point)" + n for n in names) + "};\n"
                   "int main(void) {\n  int64_t bytes = -1;\n"
                   "  if (train_embed_grad_workspace(100, 10, 8, &bytes) != LAMB_OK) return 1;\n"
                   "  if (train_embed_grad_workspace(-1, 10, 8, &bytes) != LAMB_ERR_INVALID)"
                   " return 2;\n"
                   "  printf(\"%d %d\\n\", (int)(sizeof points / sizeof points[0]),"
                   " bytes >= 0);\n  return 0;\n}\n")
    exe = tmp_path / "client"
    lib = og.library_path()
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic",
                    "-I", os.path.dirname(HEADER), str(src), "-o", str(exe), lib,
                    "-Wl,-rpath," + os.path.dirname(lib)], check=True, capture_output=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    assert out == [str(len(names)), "1"]


INVALID, ALIGN = _lib.LAMB_ERR_INVALID, _lib.LAMB_ERR_ALIGN
P = 4096  # an address that the checks accept and nothing reads


def embed_args(**change):
    a = dict(table=P, table_dtype=0, n_rows=4, dim=8, table_stride=8, ids=P, ids_dtype=1, n_ids=2,
             first_row=0, scale=1.0, out=P, out_dtype=0, out_stride=8, stream=None)
    assert set(change) <= set(a)
    return list({**a, **change}.values())


@pytest.mark.parametrize("change,code", [
    (dict(table=None), INVALID), (dict(ids=None), INVALID), (dict(out=None), INVALID),
    (dict(table_dtype=3), INVALID), (dict(out_dtype=-1), INVALID), (dict(ids_dtype=2), INVALID),
    (dict(n_rows=-1), INVALID), (dict(dim=-1), INVALID), (dict(n_ids=-1), INVALID),
    (dict(n_rows=1 << 31), INVALID), (dict(n_ids=1 << 31), INVALID),
    (dict(dim=1 << 31, table_stride=1 << 31, out_stride=1 << 31), INVALID),
    (dict(table_stride=7), INVALID), (dict(out_stride=7), INVALID),
    (dict(first_row=-1), INVALID),
    (dict(table=P + 1), ALIGN), (dict(out=P + 1), ALIGN), (dict(ids=P + 4), ALIGN),
    (dict(table=P + 2, table_dtype=2), ALIGN), (dict(out=P + 2, out_dtype=2), ALIGN),
    (dict(ids=P + 2, ids_dtype=0), ALIGN),
])
def test_embed_refuses(change, code):
    lib = og.load()
    assert lib.train_embed(*embed_args(**change)) == code
    assert lib.lamb_last_error()


def grad_args(**change):
    a = dict(grad_out=P, grad_out_dtype=0, grad_out_stride=8, ids=P, ids_dtype=1, n_ids=2,
             first_row=0, padding_id=-1, scale=1.0, accumulate=0, grad=P, grad_dtype=0, n_rows=4,
             dim=8, grad_stride=8, workspace=P, workspace_bytes=1 << 40, stream=None)
    assert set(change) <= set(a)
    return list({**a, **change}.values())


@pytest.mark.parametrize("change,code", [
    (dict(grad_out=None), INVALID), (dict(ids=None), INVALID), (dict(grad=None), INVALID),
    (dict(grad_out_dtype=3), INVALID), (dict(grad_dtype=-1), INVALID),
    (dict(ids_dtype=2), INVALID), (dict(accumulate=2), INVALID), (dict(first_row=-1), INVALID),
    (dict(n_rows=-1), INVALID), (dict(n_ids=-1), INVALID), (dict(dim=-1), INVALID),
    (dict(grad_out_stride=7), INVALID), (dict(grad_stride=7), INVALID),
    (dict(n_rows=1 << 31), INVALID), (dict(n_ids=1 << 31), INVALID),
    (dict(workspace_bytes=-1), INVALID),
    (dict(grad_out=P + 1), ALIGN), (dict(grad=P + 1), ALIGN), (dict(ids=P + 4), ALIGN),
    (dict(grad=P + 2, grad_dtype=2), ALIGN),
])
def test_embed_grad_refuses(change, code):
    lib = og.load()
    assert lib.train_embed_grad(*grad_args(**change)) == code
    assert lib.lamb_last_error()


def test_embed_grad_refuses_a_workspace_that_is_missing_small_or_misaligned():
    lib = og.load()
    need = ctypes.c_int64()
    n, rows, dim = 100_000, 1000, 64
    assert lib.train_embed_grad_workspace(n, rows, dim, ctypes.byref(need)) == _lib.LAMB_OK
    sizes = dict(n_ids=n, n_rows=rows, dim=dim, grad_out_stride=dim, grad_stride=dim)
    if need.value == 0:
        pytest.skip("no workspace is used")
    assert lib.train_embed_grad(*grad_args(workspace_bytes=need.value - 1, **sizes)) == INVALID
    assert lib.train_embed_grad(*grad_args(workspace=None, **sizes)) == INVALID
    assert lib.train_embed_grad(*grad_args(workspace=P + 8, **sizes)) == ALIGN
    assert lib.train_embed_grad_workspace(n, rows, dim, None) == INVALID
    for bad in ((-1, 1, 1), (1, -1, 1), (1, 1, -1), (1 << 31, 1, 1), (1, 1 << 31, 1)):
        assert lib.train_embed_grad_workspace(*bad, ctypes.byref(need)) == INVALID


def test_clip_create_refuses():
    lib = og.load()
    h = ctypes.c_void_p()
    one64 = lambda x: np.array([x], np.int64)
    one32 = lambda x: np.array([x], np.int32)
    ptr = lambda x: (ctypes.c_void_p * 1)(x)

    def create(n=1, sizes=one64(8), types=one32(0), grads=ptr(P), outs=None, out_types=None,
               out=ctypes.byref(h)):
        at = lambda a: None if a is None else a.ctypes.data
        return lib.train_clip_create(out, n, at(sizes), at(types), grads, outs, at(out_types),
                                     None)

    assert create(out=None) == INVALID
    assert create(n=-1) == INVALID
    assert create(sizes=None) == INVALID
    assert create(types=None) == INVALID
    assert create(grads=None) == INVALID
    assert create(sizes=one64(-1)) == INVALID
    assert create(types=one32(3)) == INVALID
    assert create(grads=ptr(None)) == INVALID
    assert create(grads=ptr(P + 1)) == ALIGN
    assert create(types=one32(2), grads=ptr(P + 2)) == ALIGN
    assert create(outs=ptr(P)) == INVALID                                  # no out types
    assert create(outs=ptr(None), out_types=one32(0)) == INVALID
    assert create(outs=ptr(2 * P + 1), out_types=one32(0)) == ALIGN
    assert create(outs=ptr(P), out_types=one32(1)) == INVALID              # itself, other type
    assert not h.value


@pytest.mark.parametrize("size", [1 << 50, (1 << 60) - 1, 1 << 62])
def test_clip_create_refuses_sizes_beyond_any_memory_at_once(size):
    # More than a table of 2^30 pieces can name; nothing is laid out for it.
    lib, h = og.load(), ctypes.c_void_p()
    sizes, types = np.array([64, size], np.int64), np.zeros(2, np.int32)
    rc = lib.train_clip_create(ctypes.byref(h), 2, sizes.ctypes.data, types.ctypes.data,
                               (ctypes.c_void_p * 2)(P, 4 * P), None, None, None)
    assert rc == INVALID and not h.value
    assert "too" in lib.lamb_last_error().decode()


def test_clip_calls_refuse_a_missing_handle():
    lib = og.load()
    assert lib.train_clip_norm(None, 1.0, P) == INVALID
    assert lib.train_clip_grads(None, 1.0, 1.0, P) == INVALID
    assert lib.train_clip_partial(None, P) == INVALID
    assert lib.train_clip_finish(None, P, 1.0, 1.0, P) == INVALID
    assert lib.train_clip_destroy(None) == _lib.LAMB_OK


def test_python_refuses_tensors_that_are_not_on_a_gpu():
    ids = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError):
        og.embed(torch.zeros(4, 8), ids)
    with pytest.raises(ValueError):
        og.embed_grad(torch.zeros(3, 8), ids, n_rows=4)
    with pytest.raises(ValueError):
        og.GradClip([torch.zeros(3)])
