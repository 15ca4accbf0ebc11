"""The serving entry points' host side, without a GPU: bad arguments come
back as status codes, never as a crash, and the C structures have the layout
that the Python binding marshals."""
import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_null_arguments_are_refused(afx):
    lib, E = afx._lib, afx.AFX_E_ARG
    size = ctypes.c_uint64(7)
    assert lib.afx_kv_tables(16, 4, None, None, 1, None, 1, None, None, None, None, None, None, 0, None, None) == E
    assert lib.afx_kv_write(None, None, None, 0, 0, None, 1, None, None) == E
    assert lib.afx_attention_workspace(None, ctypes.byref(size)) == E
    assert lib.afx_attention_plan(None, None, 0, None, None) == E
    assert lib.afx_attention(None, None, 0, 0, None, 0, 0, None, None, 0, None, None) == E
    assert lib.afx_sample(None, 2, 1, 10, 10, None, None, None, None, None, None, None, None) == E
    assert size.value == 7  # untouched on an error
    assert "null" in afx.afx_last_error() or "device memory" in afx.afx_last_error()


@pytest.mark.parametrize("page", [0, 1, 8, 24, 512])
def test_page_sizes_outside_the_list_are_refused(afx, page):
    assert afx._lib.afx_kv_tables(page, 4, None, None, 1, None, 1, None, None, None, None, None, None, 0, None,
                                  None) == afx.AFX_E_ARG
    assert "pages hold" in afx.afx_last_error()


def test_host_memory_is_refused(afx):
    buf = (ctypes.c_int32 * 64)()
    p = ctypes.addressof(buf)
    assert afx._lib.afx_kv_tables(16, 4, p, p, 1, p, 1, p, p, p + 4, p, p, p, 4, None, None) == afx.AFX_E_ARG
    assert afx._lib.afx_sample(p, 2, 1, 8, 8, None, None, None, None, p, p, None, None) == afx.AFX_E_ARG


def test_no_rows_and_no_tokens_are_no_work(afx):
    assert afx._lib.afx_sample(None, 2, 0, 10, 10, None, None, None, None, None, None, None, None) == afx.AFX_OK


def test_structures_have_the_header_s_layout(afx, tmp_path):
    gcc = shutil.which("gcc")
    if not gcc:
        pytest.skip("gcc not available")
    src = tmp_path / "layout.c"
    fields = [("afx_kv_cache", f) for f, _ in afx.afx_kv_cache._fields_]
    fields += [("afx_attention_args", f) for f, _ in afx.afx_attention_args._fields_]
    lines = ['#include "afx.h"', "#include <stddef.h>", "#include <stdio.h>", "int main(void) {",
             'printf("%zu %zu\\n", sizeof(afx_kv_cache), sizeof(afx_attention_args));']
    lines += [f'printf("%zu\\n", offsetof({s}, {f}));' for s, f in fields]
    lines += ['printf("%d %d %d %d %d\\n", AFX_KV_MAX_REQUESTS, AFX_SAMPLE_MAX_VOCAB, AFX_LOGITS_BF16, AFX_LOGITS_FP16, '
              'AFX_LOGITS_F32);',
              'printf("%d %d %d %d\\n", AFX_DEV_NO_PAGES, AFX_DEV_BAD_LENGTH, AFX_DEV_BAD_PAGE, AFX_DEV_BAD_PLAN);',
              "return 0; }"]
    src.write_text("\n".join(lines))
    exe = str(tmp_path / "layout")
    subprocess.run([gcc, "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    got = subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split()
    want = [ctypes.sizeof(afx.afx_kv_cache), ctypes.sizeof(afx.afx_attention_args)]
    want += [getattr(getattr(afx, s), f).offset for s, f in fields]
    want += [afx.AFX_KV_MAX_REQUESTS, afx.AFX_SAMPLE_MAX_VOCAB, afx.AFX_LOGITS_BF16, afx.AFX_LOGITS_FP16, afx.AFX_LOGITS_F32]
    want += [afx.AFX_DEV_NO_PAGES, afx.AFX_DEV_BAD_LENGTH, afx.AFX_DEV_BAD_PAGE, afx.AFX_DEV_BAD_PLAN]
    assert [int(x) for x in got] == want
