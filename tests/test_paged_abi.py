"""Host-side refusals of the paged cache and the logits entry points, before any device is touched."""
import ctypes

import pytest

from cross_token_latent_b200 import lib
from cross_token_latent_b200.rlt import LogitsArgs, PagedBatchArgs


def test_null_handles_and_batches_are_rejected():
    L = lib()
    p, a = PagedBatchArgs(1, 1, 1, 1, 0, 0, 0, 1, 16, 1, 1), LogitsArgs()
    ref = ctypes.byref(p)
    assert L.rlt_page_pool_bytes(None, 4, 16, 2) == 0
    assert L.rlt_paged_attention_workspace_bytes(None, ref, 4) == 0
    assert L.rlt_encode_chunk_workspace_bytes(None, ref) == 0
    for batch in (None, ref):
        assert L.rlt_paged_append(None, batch, None, None, 0, None, 0, None, 0, 0, None, 0, 0, None) == 1
        assert L.rlt_paged_attention(None, batch, None, None, 0, 1, None, 0, 0.0, None, 0, None) == 1
        assert L.rlt_encode_chunk(None, batch, None, None, None, None, 1, None, 0, None) == 1
    for args in (None, ctypes.byref(a)):
        assert L.rlt_process_logits(None, args, 1, None) == 1


def test_the_structures_have_the_header_s_layout(tmp_path):
    """sizeof and offsets as the C compiler sees them."""
    import shutil
    import subprocess
    from pathlib import Path

    if not shutil.which("gcc"):
        pytest.skip("no C compiler")
    fields = {"rlt_paged_batch": PagedBatchArgs, "rlt_logits": LogitsArgs}
    src = ['#include <stdio.h>', '#include <stddef.h>', '#include "rlt.h"', "int main(void) {"]
    for name, cls in fields.items():
        src.append(f'printf("%zu\\n", sizeof({name}));')
        src += [f'printf("%zu\\n", offsetof({name}, {f[0]}));' for f in cls._fields_]
    src.append("return 0; }")
    (tmp_path / "a.c").write_text("\n".join(src))
    inc = Path(__file__).resolve().parent.parent / "include"
    subprocess.run(["gcc", "-I", str(inc), str(tmp_path / "a.c"), "-o", str(tmp_path / "a")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "a")], capture_output=True, text=True, check=True).stdout.split()]
    want = []
    for cls in fields.values():
        want.append(ctypes.sizeof(cls))
        want += [getattr(cls, f[0]).offset for f in cls._fields_]
    assert got == want
