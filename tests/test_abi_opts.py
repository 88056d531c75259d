"""attn_opts stays what callers built earlier pass: 96 bytes, the fields where they were.
sink_tokens lies in what was padding, so that the library never reads behind a
struct of that size."""
import ctypes
import os
import subprocess

import pytest

import attention_forward_13_gb300 as A
from attention_forward_13_gb300 import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Earlier(ctypes.Structure):
    """The options before first tokens could stay visible."""
    _fields_ = [("scale", ctypes.c_float), ("causal", ctypes.c_int), ("softcap", ctypes.c_float),
                ("sink", ctypes.c_void_p), ("use_window", ctypes.c_int),
                ("window_left", ctypes.c_int), ("window_right", ctypes.c_int),
                ("top_left", ctypes.c_int), ("alibi_slopes", ctypes.c_void_p),
                ("alibi_stride", ctypes.c_int), ("bias", ctypes.c_void_p),
                ("bias_strides", _lib.attn_strides), ("scale_p", ctypes.c_float),
                ("scale_o", ctypes.c_float)]


def test_the_layout_is_the_earlier_one():
    assert ctypes.sizeof(_lib.attn_opts) == ctypes.sizeof(Earlier) == 96
    for name, _ in Earlier._fields_:
        assert getattr(_lib.attn_opts, name).offset == getattr(Earlier, name).offset, name
    at = _lib.attn_opts.sink_tokens
    for name, _ in Earlier._fields_:  # in none of the earlier fields
        f = getattr(Earlier, name)
        assert at.offset + at.size <= f.offset or at.offset >= f.offset + f.size, name


def test_the_header_agrees(tmp_path):
    src = tmp_path / "opts.c"
    lines = ["_Static_assert(offsetof(attn_opts, %s) == %d, \"%s\");" % (n, getattr(_lib.attn_opts, n).offset, n)
             for n, _ in _lib.attn_opts._fields_]
    src.write_text('#include "attn_fwd.h"\n#include <stddef.h>\n_Static_assert(sizeof(attn_opts) == 96, "size");\n' +
                   "\n".join(lines) + "\n")
    subprocess.run(["gcc", "-std=c11", "-fsyntax-only", "-I", os.path.join(ROOT, "include"), str(src)], check=True)


@pytest.mark.parametrize("behind", [0x00, 0x01, 0x7F, 0xFF])
def test_nothing_behind_an_earlier_struct_is_read(behind):
    """An earlier caller's struct with other memory right behind it: the same schedule."""
    def schedule(after):
        buf = ctypes.create_string_buffer(bytes([after]) * 128, 128)
        o = Earlier.from_buffer(buf)
        ctypes.memset(ctypes.addressof(o), 0, ctypes.sizeof(o))
        o.causal, o.use_window, o.window_left, o.window_right = 1, 1, 500, -1
        off, item = (ctypes.c_int32 * 101)(), (ctypes.c_int32 * 4096)()
        st = A.library().attn_dense_schedule(2, 8, 8, 4096, 4096, ctypes.cast(buf, ctypes.POINTER(_lib.attn_opts)), 100,
                                             off, item)
        return st, list(off), list(item)

    assert schedule(behind) == schedule(0)
