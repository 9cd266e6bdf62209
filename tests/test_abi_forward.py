"""Host-side refusals of the paged, attention and logits entry points that need no GPU: a null handle is refused before
any argument is looked at, and the binding's structures have the header's layout."""
import ctypes
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def libdt():
    import __graft_entry__

    __graft_entry__._load_builder().build()
    from dynamic_draft_tree_gb300 import _lib

    return _lib


def test_null_handle_is_refused(libdt):
    lib, bad = libdt.lib, libdt.DT_ERR_ARG
    n = ctypes.c_int64(0)
    assert lib.dt_kv_reserve(None, 1, None, None, None, 0, None, 0, 1, None, None) == bad
    assert lib.dt_kv_release(None, 1, None, None, None) == bad
    assert lib.dt_commit_kv_paged(None, 1, None, 1, None, None, 0, None, 0, None, 0, 1, None, None, None, None) == bad
    assert lib.dt_tree_attention(None, None, None) == bad
    assert lib.dt_tree_attention_workspace(None, 1, 1, 1, 1, 64, 0, ctypes.byref(n)) == bad
    assert lib.dt_count_tokens(None, 1, None, None, 0, 1, None, None, 0, None, 0, 0, None) == bad
    assert lib.dt_logits_process(None, 1, None, 0, None, 0, None, None) == bad
    assert "null" in lib.dt_last_error_string().decode()


def test_structures_match_the_header(libdt, tmp_path):
    """Sizes and offsets as the C compiler lays them out."""
    names = {"dt_block_pool": libdt.DtBlockPool, "dt_kv_rows": libdt.DtKvRows, "dt_attn_args": libdt.DtAttnArgs,
             "dt_logits_params": libdt.DtLogitsParams}
    lines = []
    for c, py in names.items():
        lines.append(f'printf("{c} %zu\\n", sizeof({c}));')
        lines += [f'printf("{c}.{f[0]} %zu\\n", offsetof({c}, {f[0]}));' for f in py._fields_]
    src = tmp_path / "s.c"
    src.write_text("#include <stddef.h>\n#include <stdio.h>\n#include \"dt.h\"\nint main(void) {\n" + "\n".join(lines)
                   + "\nreturn 0;\n}\n")
    exe = tmp_path / "s"
    subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), "-I", "/usr/local/cuda/include", str(src), "-o",
                           str(exe)])
    got = dict(x.rsplit(" ", 1) for x in subprocess.check_output([str(exe)]).decode().split("\n") if x)
    for c, py in names.items():
        assert int(got[c]) == ctypes.sizeof(py), c
        for f in py._fields_:
            assert int(got[f"{c}.{f[0]}"]) == getattr(py, f[0]).offset, (c, f[0])


def test_packed_structures_are_the_structures(libdt):
    import dynamic_draft_tree_gb300 as dt

    for cls, pack in ((libdt.DtKvRows, dt._pack_kv_rows), (libdt.DtAttnArgs, dt._pack_attn),
                      (libdt.DtLogitsParams, dt._pack_logits)):
        values = [0.5 if f[1] is ctypes.c_float else 3 * k + 1 for k, f in enumerate(cls._fields_)]
        assert pack(*values) == bytes(cls(*values))


def test_header_comments_name_every_status_bit():
    text = open(os.path.join(ROOT, "include", "dt.h")).read()
    bits = dict(re.findall(r"(DT_DEV_[A-Z_]+) = (\d+)", text))
    from dynamic_draft_tree_gb300 import _lib

    for name, value in bits.items():
        assert getattr(_lib, name) == int(value), name
