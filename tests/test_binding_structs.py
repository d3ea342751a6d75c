"""The binding's argument structs lie as the header's do, calls without a handle
are refused, and the sizes of the callers' buffers can be asked for without a
GPU."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

import exact_bpe_tokenization_utf_gb300 as pkg

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STRUCTS = {"tok_paged_args": pkg.PagedArgs, "tok_logits_args": pkg.LogitsArgs, "tok_logits_grad_args": pkg.LogitsGradArgs,
           "tok_embed_args": pkg.EmbedArgs, "tok_embed_grad_args": pkg.EmbedGradArgs, "tok_sample_args": pkg.SampleArgs,
           "tok_kv_cache": pkg.KVCache, "tok_store_args": pkg.StoreArgs, "tok_attend_args": pkg.AttendArgs}


@pytest.fixture(scope="module")
def lib():
    from exact_bpe_tokenization_utf_gb300 import _build
    _build.build()
    return pkg.lib()


def test_every_struct_of_the_header_is_bound():
    with open(os.path.join(ROOT, "include", "tok.h")) as f:
        assert sorted(re.findall(r"^\} (tok_\w+);", f.read(), re.M)) == sorted(STRUCTS)


def test_structs_lie_as_in_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if not cc:
        pytest.skip("no C compiler")
    lines = ["#include <stddef.h>", "#include <stdio.h>", '#include "tok.h"', "int main(void) {"]
    want = []
    for name, cls in STRUCTS.items():
        lines.append('  printf("%%d\\n", (int)sizeof(%s));' % name)
        want.append(ctypes.sizeof(cls))
        for field, kind in cls._fields_:
            lines.append('  printf("%%d %%d\\n", (int)offsetof(%s, %s), (int)sizeof(((%s*)0)->%s));' % (name, field, name, field))
            want.append((getattr(cls, field).offset, ctypes.sizeof(kind)))
    src, exe = tmp_path / "s.c", tmp_path / "s"
    src.write_text("\n".join(lines + ["  return 0;", "}", ""]))
    subprocess.run([cc, "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines()
    got = [tuple(map(int, x.split())) if " " in x else int(x) for x in out]
    assert got == want


def test_unknown_fields_are_refused():
    with pytest.raises(TypeError):
        pkg.SampleArgs(d_logits=1)


def test_calls_without_a_handle(lib):
    for call in (lib.tok_embed, lib.tok_embed_backward, lib.tok_sample):
        assert call(None, None, None) == pkg.TOK_EINVAL
    for call in (lib.tok_paged_store, lib.tok_paged_attend):
        assert call(None, None, None, None) == pkg.TOK_EINVAL
    assert lib.tok_paged_attend_work_bytes(None, 1, 8, 8, 64) == 0


def test_sizes_of_the_gradients_buffer(lib):
    size = lib.tok_embed_work_bytes
    assert size(1 << 31, 20, 8) == 0 and size(5, 0, 8) == 0 and size(5, (1 << 20) + 1, 8) == 0 and size(5, 5, 0) == 0
    for rows, dim in ((700, 8), (100257, 2048), (1 << 20, 256), (3, 1)):
        steps = [size(n, rows, dim) for n in list(range(0, 9000, 13)) + list(range(9000, 2000000, 1777))]
        assert steps == sorted(steps) and steps[0] > 0 and all(s % 256 == 0 for s in steps)
