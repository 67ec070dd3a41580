"""The hand-counted waits of the kernels with an adapter for every row, on the gfx950 assembly of this
repository's own sources (CPU only).

The mid kernel requests X by DMA and the codes and constants into registers two steps ahead; each step
starts with a hand-written `s_waitcnt vmcnt(N); s_barrier` that must leave exactly the requests of one
step in flight, so N must equal the vector-memory operations of a step; a wait the compiler inserted must
not retire any of the step's own. The multi forms of the large kernels keep the step of their plain forms.
"""
import re

import pytest

from tests.test_kernel_waits import check_step_pipeline, device_asm, kernels, main_loops, pytestmark, vmcnt  # noqa: F401


def test_mid_kernel_step_waits(tmp_path):
    ks = {k: b for k, b in kernels(device_asm("mid.hip", str(tmp_path))).items() if "mid_kernel" in k}
    assert len(ks) == 48     # 3 formats x 8 heights x K a multiple of the step or not
    for name, body in ks.items():
        loops = main_loops(body)
        assert len(loops) == 1, name
        steps, cur = [], None
        for kind, text, hand in loops[0]:
            if kind == "wait" and hand:
                cur = []
                steps.append((vmcnt(text), cur))
            elif cur is not None:
                cur.append((kind, text))
        assert len(steps) == 3, (name, len(steps))     # three buffers
        for n, ops in steps:
            loads = [t for k, t in ops if k == "mem"]
            assert len(loads) == n, (name, n, len(loads))
            assert any(t.endswith(" lds") for t in loads), name
            seen = 0
            for k, t in ops:
                seen += k == "mem"
                assert k == "mem" or vmcnt(t) >= seen, (name, t)


@pytest.mark.parametrize("src,pattern", [("fwd.hip", "fwd_multi_kernel"), ("dx.hip", "dx_multi_kernel"),
                                         ("dx.hip", "dx_split_kernel")])
def test_large_kernel_step_waits(tmp_path, src, pattern):
    ks = {k: b for k, b in kernels(device_asm(src, str(tmp_path))).items() if pattern in k}
    assert len(ks) == (9 if pattern == "dx_split_kernel" else 3)     # 3 formats, the split at 3 heights
    for name, body in ks.items():
        loops = main_loops(body)
        assert len(loops) == 1, name
        check_step_pipeline(name, loops[0])


def test_stream_kernel_multi_form(tmp_path):
    """The copying waves' loop holds hand-issued copies and hand waits only."""
    ks = {k: b for k, b in kernels(device_asm("decode16.hip", str(tmp_path))).items() if "stream16_multi" in k}
    assert len(ks) == 2
    for name, body in ks.items():
        copying = [s for s in main_loops(body) if any(k == "mem" and t.endswith(" lds") for k, t, a in s)]
        assert len(copying) == 1, name
        assert all(a for k, t, a in copying[0]), name
        assert re.search("ILb[01]E", name)
