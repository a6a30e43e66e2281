"""The cache calls' host side at the edges of what their documentation allows (no GPU needed)."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("capturing", [True, False])
def test_a_new_workspace_clears_its_state_only(monkeypatch, capturing):
    """The calls of a captured round clear their workspaces in every replay: status word and counters, not the partial results."""
    from speculative_decoding_verify_temperature_b200 import build, kv_cache
    build.build()
    header = open(os.path.join(ROOT, "include", "spec_verify.h")).read()
    state = int(re.search(r"#define SPEC_CACHE_STATE_BYTES (\d+)", header).group(1))
    cleared = []
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: capturing, raising=False)
    monkeypatch.setattr(kv_cache, "spec_workspace_init", lambda buf: cleared.append((buf.data_ptr(), buf.numel())))
    monkeypatch.setattr(kv_cache, "_cache_ws", {})
    ws = kv_cache._workspace(None, torch.device("cpu"), 0, 4, 64, 64, 128)
    assert ws.numel() >= kv_cache.spec_cache_workspace_bytes(4, 64, 64, 128) > 30 << 20
    assert cleared == [(ws.data_ptr(), state)]


@pytest.mark.parametrize("axis", range(3))
@pytest.mark.parametrize("which", ["q_out", "k_out"])
def test_norm_rope_refuses_outputs_that_overlap_themselves(axis, which):
    """A broadcast output would be written by several CTAs at once."""
    from speculative_decoding_verify_temperature_b200 import build, spec_verify as sv
    build.build()
    L, fake = sv.lib(), 1 << 20

    def call(strides):
        rows = {n: [12 * 64, 4 * 64, 64] for n in ("q", "k", "q_out", "k_out")}
        rows[which] = strides
        q, k, qo, ko = ((ctypes.c_int64 * 3)(*rows[n]) for n in ("q", "k", "q_out", "k_out"))
        return L.spec_qk_norm_rope(2, 3, 4, 4, 64, fake, q, fake, k, 1, fake, fake, 64, 0, None, None, 1, 1e-6, fake, qo, fake, ko,
                                   None)

    for stride in (0, 32, 56):
        strides = [12 * 64, 4 * 64, 64]
        strides[axis] = stride
        assert call(strides) == sv.SPEC_ERR_INVALID_ARG
        assert which in L.spec_last_error_detail().decode()


def test_a_cache_keeps_its_tensors():
    """The library holds their addresses: assigning another tensor would leave it with the old one's memory."""
    import speculative_decoding_verify_temperature_b200 as spec
    from test_cache_host import _tensors
    c = spec.KvCache(**_tensors())
    for name in ("k_pages", "v_scale", "k_open", "page_table", "lengths", "slots", "head_dim"):
        was = getattr(c, name)
        with pytest.raises(AttributeError, match="batch"):
            setattr(c, name, was)
        assert getattr(c, name) is was
    d = c.batch(c.page_table[:1], c.lengths[:1].clone())
    assert d.B == 1 and d.k_pages is c.k_pages and d.lengths is not c.lengths
