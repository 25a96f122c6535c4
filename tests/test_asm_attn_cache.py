"""The copies into LDS of the attention over the cache are inline asm, whose
hazards the compiler does not see: M0 holds the LDS address and has to be written
by the scalar unit, at least one wait state (the asm's own s_nop) before the
copy, and nothing may write it in between."""
import os
import re
import subprocess

from async_tensor_tile_amd import _build


def test_lds_copies_have_their_wait_state(tmp_path):
    out = str(tmp_path / "attn.s")
    subprocess.check_call([_build.HIPCC, *_build.FLAGS, "--cuda-device-only", "-S",
                           os.path.join(_build.CSRC, "kernel_attn_cache_bf16_same.hip"), "-o", out],
                          stderr=subprocess.DEVNULL)
    with open(out) as f:
        lines = [l.split(";", 1)[0].strip() for l in f]
    lines = [l for l in lines if l]
    copies = [i for i, l in enumerate(lines) if l.startswith("global_load_lds_dwordx4")]
    assert copies
    for i in copies:
        assert re.match(r"global_load_lds_dwordx4 v\[\d+:\d+\], off$", lines[i]), lines[i]
        assert re.match(r"s_nop [0-9]+$", lines[i - 1]), lines[i - 1]
    for l in lines:
        if re.search(r"\bm0\b", l) and not l.startswith("global_load_lds"):
            assert re.match(r"s_(mov|add|or|lshl|and|addk|movk|sub|lshl_add)\w* m0,", l) or ", m0" in l, l
