"""Host-side refusals of the prompt attention, log probability and fork entry points that need no GPU, and the layout of the
binding's structures."""
import ctypes
import os
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
    assert lib.dt_prompt_attention(None, None, None) == bad
    assert lib.dt_prompt_attention(None, bytes(libdt.DtPromptArgs()), None) == bad
    assert lib.dt_prompt_attention_workspace(None, 1, 1, 1, 64, ctypes.byref(n)) == bad
    assert lib.dt_token_logprobs(None, None, 0, None, None) == bad
    assert lib.dt_token_logprobs(None, None, 0, bytes(libdt.DtLogprobArgs()), None) == bad
    assert lib.dt_token_logprobs_workspace(None, 1, 0, ctypes.byref(n)) == bad
    assert lib.dt_kv_fork(None, 1, None, None, None, 1, None, None, None, None, 0, None) == bad
    assert lib.dt_kv_release_shared(None, 1, None, None, None, None) == bad
    assert "null" in lib.dt_last_error_string().decode() and n.value == 0


def test_structures_match_the_header(libdt, tmp_path):
    names = {"dt_prompt_args": libdt.DtPromptArgs, "dt_logprob_args": libdt.DtLogprobArgs, "dt_kv_pages": libdt.DtKvPages}
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

    for cls, pack in ((libdt.DtPromptArgs, dt._pack_prompt), (libdt.DtLogprobArgs, dt._pack_logprobs),
                      (libdt.DtKvPages, dt._pack_kv_pages)):
        values = [0.5 if f[1] is ctypes.c_float else 3 * k + 1 for k, f in enumerate(cls._fields_)]
        assert pack(*values) == bytes(cls(*values))


def test_entry_points_are_exported(libdt):
    for name in ("dt_prompt_attention", "dt_prompt_attention_workspace", "dt_token_logprobs", "dt_token_logprobs_workspace",
                 "dt_kv_fork", "dt_kv_release_shared"):
        assert name in libdt.EXPORTS and hasattr(libdt.lib, name)
